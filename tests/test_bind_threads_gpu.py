"""While a rotary or paged call is inside the library (a launch waits when the
stream's queue is full), other Python threads run, as with the dense calls."""
import ctypes
import subprocess
import threading
import time

import pytest
import torch

from attention_swa_forward_gb300 import swa
from tests.test_paged_order_gpu import MIXED, Serving
from tests.test_paged_refusals_gpu import APPEND_ROPE, D, N, N_KV, T, append_args, forward_args, geometry, zeros

pytestmark = pytest.mark.gpu
WAIT = 0.4  # seconds


@pytest.fixture(scope="module")
def slow_entry(tmp_path_factory):
    """The address of an entry point that takes WAIT seconds and does nothing."""
    d = tmp_path_factory.mktemp("slow")
    (d / "slow.c").write_text(f"#include <unistd.h>\nint slow() {{ usleep({int(WAIT * 1e6)}); return 0; }}\n")
    subprocess.run(["gcc", "-shared", "-fPIC", str(d / "slow.c"), "-o", str(d / "slow.so")], check=True)
    lib = ctypes.CDLL(str(d / "slow.so"))
    return ctypes.cast(lib.slow, ctypes.c_void_p).value


def test_other_threads_run_during_a_call(slow_entry, monkeypatch):
    geom, args, more = geometry(), forward_args(), append_args()
    q, k, pos = zeros(T, N, D), zeros(T, N_KV, D), zeros(2, T, dtype=torch.int32)
    calls = {
        "rope": lambda: swa.rope(APPEND_ROPE, q, k, pos),
        "append": lambda: swa.paged_append(geom, rope=APPEND_ROPE, **more),
        "forward": lambda: swa.paged_forward(geom, **args),
    }
    for call in calls.values():
        call()
    torch.cuda.synchronize()
    monkeypatch.setattr(swa.lib(), "entries", dict.fromkeys(swa.lib().entries, slow_entry))
    for name, call in calls.items():
        ticks, done = [], threading.Event()

        def watch():
            while not done.is_set():
                ticks.append(time.monotonic())
                time.sleep(0.01)

        other = threading.Thread(target=watch)
        other.start()
        try:
            t0 = time.monotonic()
            call()
            t1 = time.monotonic()
        finally:
            done.set()
            other.join()
        assert t1 - t0 >= WAIT * 0.9
        # a thread that sleeps 10 ms at a time ran through the middle of the call
        assert sum(t0 + 0.25 * WAIT < t < t0 + 0.75 * WAIT for t in ticks) >= 3, name


def test_a_stream_that_is_no_handle_enqueues_nothing():
    out = torch.full((T, N, D), 7.0, dtype=torch.bfloat16, device="cuda:0")
    args = {**forward_args(), "out": out}

    class Odd:
        cuda_stream = "no handle"

    with pytest.raises(ValueError, match="stream"):
        swa.paged_forward(geometry(), **args, workspace=swa.paged_forward_workspace(geometry(), "cuda:0"), stream=Odd())
    torch.cuda.synchronize()
    assert (out == 7).all()


@pytest.mark.parametrize("one_stream", [True, False])
def test_threads_that_call_at_once_match_serial_calls(one_stream):
    """Mixed batches, whose calls are up to four launches, from four threads: their
    launches interleave, on one stream or on four; each has its own workspaces."""
    names = ["40_tiles_split", "40_few_rows_joined", "40_last_round_split", "17_tiles_of_a_round"]
    work = []
    for i, name in enumerate(names):
        s = Serving(*MIXED[name](), 23 + i)
        s.feed()
        s.step()
        work.append((s, s.check(name)))
    torch.cuda.synchronize()
    shared = torch.cuda.Stream()
    got, errors = [[] for _ in work], []
    start = threading.Barrier(len(work))

    def run(i):
        try:
            s = work[i][0]
            with torch.cuda.stream(shared if one_stream else torch.cuda.Stream()):
                start.wait()
                for _ in range(40):
                    for t in (s.rq, s.out, s.sm, s.ss):
                        t.fill_(7.0)
                    s.step()
                    got[i].append([t.clone() for t in (s.out, s.sm, s.ss)])
        except Exception as e:  # noqa: BLE001 (raised below, in the test's thread)
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for (s, want), res in zip(work, got):
        assert len(res) == 40
        for again in res:
            for a, b in zip(want, again):
                assert torch.equal(a, b)
