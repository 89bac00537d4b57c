"""pkv_device_error over the check words of several translation units: one call reports a code and clears
every word, and calls from several threads do not disturb one another."""
import threading

import pytest
import torch

from paged_kv_cache_73_gb300 import binding as pkv

pytestmark = pytest.mark.gpu

B, H, D = 16, 2, 64


def _bad_slot(dev):
    pool = torch.zeros(pkv.int4_cache_shape(2, H, B, D), dtype=torch.uint8, device=dev)
    x = torch.zeros(1, H, D, dtype=torch.float16, device=dev)
    pkv.reshape_and_cache_int4(x, x, pool, pool.clone(), torch.tensor([2 * B], device=dev), B)


def _bad_pair(dev):
    pool = torch.zeros(2, H, B, D, dtype=torch.float16, device=dev)
    pkv.copy_blocks([pool], [pool.clone()], torch.tensor([[0, 2]], device=dev))


def test_codes_of_two_units(cuda_device):
    assert pkv.device_error() == 0
    _bad_slot(cuda_device)
    _bad_pair(cuda_device)
    assert pkv.device_error(reset=False) in (3, 4) and pkv.device_error(reset=False) in (3, 4)
    assert pkv.device_error() in (3, 4)
    assert pkv.device_error() == 0                           # both words are clear


def test_a_stream_of_its_own(cuda_device):
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        _bad_slot(cuda_device)
    assert pkv.device_error(stream=st) == 3 and pkv.device_error(stream=st) == 0


def test_many_threads_at_once(cuda_device):
    seen, failures = [], []

    def check():
        try:
            st = torch.cuda.Stream()
            for _ in range(50):
                seen.append(pkv.device_error(stream=st))
        except Exception as e:                               # noqa: BLE001 - reported below
            failures.append(e)

    _bad_slot(cuda_device)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=check) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures and len(seen) == 400
    assert 3 in seen and set(seen) <= {0, 3} and pkv.device_error() == 0
