"""Handle-free calls of two host threads at a time, with sizes that want different amounts of shared
memory: neither call may fail because of the other's (ctypes lets the threads run side by side)."""
import threading

import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu
CALLS = 4000


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32, device="cuda")


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device="cuda")


def side_by_side(works):
    """Runs each work CALLS times on a thread and a stream of its own; the errors."""
    errors, start = [], threading.Barrier(len(works))

    def run(work, stream):
        torch.cuda.synchronize()
        start.wait()
        try:
            for _ in range(CALLS):
                work(stream)
        except Exception as e:
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(w, torch.cuda.Stream())) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


def test_products_of_different_numbers_of_groups():
    def product(G):
        a, sa, counts, offs = u8(128, 16), u8(512), i32(G), i32(G + 1)
        counts[0] = 3
        a.fill_(0x22)                       # ones
        sa.fill_(127)
        w, sw, out = u8(G, 32, 16).fill_(0x44), u8(G * 512).fill_(127), torch.zeros(128, 32, device="cuda")

        def work(stream):
            moe.moe_grouped_gemm_mxfp4(a, sa, counts, offs, w, sw, out, stream=stream)
        return work, out

    many, few = product(600), product(1)
    assert not side_by_side([many[0], few[0]])
    for _, out in (many, few):
        assert torch.all(out[:3] == 64.0) and torch.all(out[3:] == 0.0)


@pytest.mark.parametrize("T", [512, 1024])   # one launch; the sort's own
def test_sorts_of_different_numbers_of_experts(T):
    def dispatch(E):
        ids = (torch.arange(2 * T, device="cuda", dtype=torch.int32) % E).view(T, 2).contiguous()
        counts, offs, perm, inv = i32(E), i32(E + 1), i32(2 * T), i32(2 * T)

        def work(stream):
            moe.moe_dispatch(None, ids, E, 0, E, 1, counts, offs, perm, inv, None, stream=stream)
        return work, ids, counts, inv

    both = [dispatch(1024), dispatch(320)]
    assert not side_by_side([b[0] for b in both])
    for _, ids, counts, inv in both:
        assert torch.equal(counts.long(), torch.bincount(ids.view(-1).long(), minlength=counts.numel()))
        want = torch.empty_like(inv, dtype=torch.int64)
        want[torch.argsort(ids.view(-1).long(), stable=True)] = torch.arange(2 * T, device="cuda")
        assert torch.equal(inv.long(), want)
