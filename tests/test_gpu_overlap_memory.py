"""The overlapped calls' memory: what a waiting layout still reads and writes."""
import pytest
import torch

from combine_get_dispatch_layout_amd import ep

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,E,K,H", [(4000, 8, 2, 64), (200, 64, 8, 2048), (700, 128, 8, 256)])
def test_dropped_layout_outputs_are_not_written_over(N, E, K, H):
    """A caller that keeps neither the outputs nor the ids of the next batch: the
    combine must not write into memory that was given out again, and lays out
    what was asked for."""
    print(f"[overlap memory] {N} {E} {K}", flush=True)
    cfg = ep.Config(hidden=H, num_topk=K, num_experts=E, num_ranks=2)
    h, nxt, other = (ep.ep_handle_init(cfg, N) for _ in range(3))
    idx = torch.rand((N, E), device="cuda").topk(K, dim=1).indices.int()
    want = ep.ep_get_layout(other, idx)
    ep.ep_get_layout(h, idx)
    rows = ep.ep_recv_capacity(cfg, N)
    x = torch.randn((N, H), device="cuda").to(torch.bfloat16)
    recv, out, w = torch.empty((rows, H), dtype=x.dtype, device="cuda"), torch.empty_like(x), torch.ones((N, K), device="cuda")
    torch.cuda.synchronize()
    ep.ep_dispatch_overlap(h, x, recv, h_next=nxt, topk_next=idx.clone())
    taken = [torch.full_like(t, 1) for t in want.values() if t is not None for _ in range(3)]
    taken += [torch.full_like(idx, 1) for _ in range(3)]
    ep.ep_combine_overlap(h, recv, w, out, h_next=nxt)
    torch.cuda.synchronize()
    assert all((t == 1).all() for t in taken)
    a, b = ep.ep_handle_view(nxt), ep.ep_handle_view(other)
    for k in ("psum_expert", "num_unaligned", "slot_idx", "topk_idx"):
        if k in b:
            assert torch.equal(a[k], b[k]), k
    assert nxt._waiting is None
    assert ep.ep_check_error(nxt) == (ep.EP_OK, 0)
