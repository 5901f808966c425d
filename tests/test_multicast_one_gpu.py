"""The multicast option is for jobs of one GPU: the handle and the benchmark refuse it in a job of
several ranks, before anything touches a GPU."""
import os
import socket
import subprocess
import sys

import pytest
import torch.multiprocessing as mp

from mixture_experts_layer_16_gb300 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHAPE = (64, 256, 128, 8, 2)


def test_shape_in_a_job_of_two_ranks(monkeypatch):
    monkeypatch.setenv("WORLD_SIZE", "2")
    with pytest.raises(ValueError, match="one GPU"):
        B.make_shape(*SHAPE, multicast=True)
    assert B.make_shape(*SHAPE).flags == 0
    for alone in ("1", ""):
        monkeypatch.setenv("WORLD_SIZE", alone)
        assert B.make_shape(*SHAPE, multicast=True).flags == B.MM_MOE_MULTICAST


def _rank(rank, port, q):
    import torch.distributed as dist
    os.environ.pop("WORLD_SIZE", None)
    dist.init_process_group("gloo", init_method=f"tcp://127.0.0.1:{port}", rank=rank, world_size=2)
    try:
        B.make_shape(*SHAPE, multicast=True)
        q.put("accepted")
    except ValueError:
        q.put("refused")
    dist.destroy_process_group()


def test_shape_under_a_process_group():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    procs = [ctx.Process(target=_rank, args=(r, port, q)) for r in range(2)]
    for p in procs:
        p.start()
    assert [q.get(timeout=120) for _ in procs] == ["refused"] * 2
    for p in procs:
        p.join(timeout=60)
        assert p.exitcode == 0


@pytest.mark.parametrize("gpus,world", [("2", "1"), ("1", "2"), ("8", "8")])
def test_benchmark_of_several_gpus(gpus, world):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--gpus", gpus, "--multicast",
                        "--config", "tiny", "--steps", "1", "--warmup", "0"], capture_output=True,
                       text=True, cwd=ROOT, timeout=120,
                       env=dict(os.environ, WORLD_SIZE=world, RANK="0", LOCAL_RANK="0"))
    assert r.returncode == 2 and "--multicast is for one GPU" in r.stderr
    assert r.stdout.strip() == ""
