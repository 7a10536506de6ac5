"""sync_status: every kernel family's sticky flags are reported once and together, at the price of few blocking copies."""
import statistics
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from nvfp4_block_scaled_07_gb300 import build
    build.build()
    from nvfp4_block_scaled_07_gb300 import binding
    binding.device_check()
    binding.sync_status()
    return binding


def _median_us(call, n=300):
    for _ in range(20):
        call()
    times = []
    for _ in range(n):
        t = time.perf_counter()
        call()
        times.append(time.perf_counter() - t)
    return statistics.median(times) * 1e6


def test_sync_status_takes_less_than_four_blocking_copies(B):
    """It read and cleared two flags with four copies before there were more kinds of kernels; with more it takes no more."""
    device, host = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32)
    torch.cuda.synchronize()
    ratios = []
    for _ in range(5):
        copy = _median_us(lambda: host.copy_(device))
        ratios.append(_median_us(B.sync_status) / copy)
    assert min(ratios) < 4, ratios


def _bad_append(mla):
    x = torch.zeros((1, 576), dtype=torch.bfloat16, device="cuda")
    mla.mla_append(x[:, :512], x[:, 512:], torch.full((1,), 99, dtype=torch.int32, device="cuda"),
                   torch.zeros(1, dtype=torch.int64, device="cuda"), mla.rope_table(4),
                   torch.zeros((1, 16, 576), dtype=torch.bfloat16, device="cuda"))


def _bad_decode(mla):
    q = torch.zeros((1, 1, 16, 576), dtype=torch.bfloat16, device="cuda")
    mla.mla_decode(q, torch.zeros((1, 16, 576), dtype=torch.bfloat16, device="cuda"),
                   torch.full((1, 1), 7, dtype=torch.int32, device="cuda"),
                   torch.ones(1, dtype=torch.int32, device="cuda"), 0.1)


def _bad_prefill(mla):
    q = torch.zeros((1, 1, 192), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    mla.mla_prefill(q, q[..., :128], q[:, 0, 128:], q[..., :128], cu, cu, 0.1)


@pytest.mark.parametrize("calls", [(_bad_append,), (_bad_decode,), (_bad_prefill,), (_bad_append, _bad_decode, _bad_prefill)])
def test_flags_are_reported_once(B, calls):
    from nvfp4_block_scaled_07_gb300 import mla
    for call in calls:
        call(mla)
    with pytest.raises(B.Nvfp4MoeError) as e:
        B.sync_status()
    assert e.value.status == B.ERR_DEVICE_DATA
    B.sync_status()


def test_a_timeout_is_told_before_bad_data_and_both_are_cleared(B):
    from nvfp4_block_scaled_07_gb300 import mla
    B.set_wait_limit_us(1000)
    try:
        _bad_append(mla)
        B.wait_selftest(expected_arrivals=2, arrivals=1)       # a bounded wait that cannot complete
        with pytest.raises(B.Nvfp4MoeError) as e:
            B.sync_status()
        assert e.value.status == B.ERR_TIMEOUT
        B.sync_status()
    finally:
        B.set_wait_limit_us(0)


def test_one_of_several_threads_gets_a_flag(B):
    """Threads that ask at once, each on a stream of its own: a flag reaches one of them, and exactly one."""
    from nvfp4_block_scaled_07_gb300 import mla
    for _ in range(20):
        _bad_append(mla)
        torch.cuda.synchronize()
        seen = []

        def ask():
            with torch.cuda.stream(torch.cuda.Stream()):
                try:
                    B.sync_status()
                except B.Nvfp4MoeError as e:
                    seen.append(e.status)
        threads = [threading.Thread(target=ask) for _ in range(4)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert seen == [B.ERR_DEVICE_DATA]
