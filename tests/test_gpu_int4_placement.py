"""Where the tensors of the four-bit path and of the prompt operators live: on the current device (refused on the
host otherwise, before any kernel runs), and, where a call allocates, on the stream it was given."""
import pytest
import torch

from paged_kv_cache_73_gb300 import binding as pkv

pytestmark = pytest.mark.gpu

B, H, D = 16, 2, 64


def calls(dev):
    """Every entry point by name: a function of keyword arguments (stream)."""
    x = torch.randn(32, H, D, device=dev).half()
    pools = [torch.zeros(pkv.int4_cache_shape(4, H, B, D), dtype=torch.uint8, device=dev) for _ in range(2)]
    slots = torch.arange(32, device=dev)
    pkv.reshape_and_cache_int4(x, x, *pools, slots, B)
    pos = torch.arange(32, dtype=torch.int32, device=dev)
    freq = pkv.rope_frequencies([1.0 / (1 + i) for i in range(D // 2)], dev)
    start = torch.tensor([0, 32], dtype=torch.int32, device=dev)
    tables = torch.tensor([[0, 1]], dtype=torch.int32, device=dev)
    lens = torch.tensor([32], dtype=torch.int32, device=dev)
    pairs = torch.tensor([[0, 2]], device=dev)
    return dict(
        qk_norm_rope=lambda **kw: pkv.qk_norm_rope(x, x, pos, freq, **kw),
        reshape_and_cache_int4=lambda **kw: pkv.reshape_and_cache_int4(x, x, *pools, slots, B, **kw),
        gather_cache_int4=lambda **kw: pkv.gather_cache_int4(*pools, slots, B, **kw),
        copy_blocks_int4=lambda **kw: pkv.copy_blocks_int4(pools[:1], pools[1:], pairs, B, **kw),
        swap_blocks_int4=lambda **kw: pkv.swap_blocks_int4(pools[:1], pools[1:], pools[:1], pools[1:], pairs, B, **kw),
        paged_attention_decode_int4=lambda **kw: pkv.paged_attention_decode_int4(x[:1], *pools, tables, lens, 0.1, B, **kw),
        prompt_attention=lambda **kw: pkv.prompt_attention(x, x, x, start, 0.1, 32, **kw))


NAMES = ["qk_norm_rope", "reshape_and_cache_int4", "gather_cache_int4", "copy_blocks_int4", "swap_blocks_int4",
         "paged_attention_decode_int4", "prompt_attention"]


@pytest.mark.parametrize("name", NAMES)
def test_another_device_is_refused(cuda_device, monkeypatch, name):
    call = calls(cuda_device)[name]
    torch.cuda.synchronize()
    # the tensors live on cuda:0; make the binding see another current device
    monkeypatch.setattr(torch.cuda, "current_device", lambda: cuda_device.index + 1)
    with pytest.raises(pkv.PkvError) as e:
        call()
    assert e.value.status == pkv.PKV_ERR_INVALID_ARG and "current CUDA device" in str(e.value)
    monkeypatch.undo()
    call()
    assert pkv.device_error() == 0


def _stream_of(t):
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the allocator's memory")


@pytest.mark.parametrize("name", ["qk_norm_rope", "gather_cache_int4", "paged_attention_decode_int4", "prompt_attention"])
def test_results_belong_to_the_stream_given(cuda_device, name):
    call = calls(cuda_device)[name]
    plain = call()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for stream in (st, st.cuda_stream):
        got = call(stream=stream)
        st.synchronize()
        for g, w in zip(got if isinstance(got, tuple) else (got,), plain if isinstance(plain, tuple) else (plain,)):
            assert _stream_of(g) == st.cuda_stream and torch.equal(g, w)
    call(stream=0)
    assert pkv.device_error() == 0


def test_workspace_elsewhere_is_refused(cuda_device):
    call = calls(cuda_device)["paged_attention_decode_int4"]
    n = pkv.paged_attention_int4_workspace_size(1, H, H, D, 2, B)
    for bad in (torch.empty(n, dtype=torch.uint8), torch.empty(n, 2, dtype=torch.uint8, device=cuda_device)[:, 0]):
        with pytest.raises(pkv.PkvError) as e:
            call(workspace=bad)
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG and "workspace" in str(e.value)
    call(workspace=torch.empty(n, dtype=torch.uint8, device=cuda_device))
    assert pkv.device_error() == 0
