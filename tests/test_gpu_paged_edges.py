"""The attention calls of include/hb_paged.h on the GPU where workspaces and
numbers are the least usual that they allow, against plain 64-bit forms
(paged_ref.py)."""
import pytest

from chunked_prefill_hybrid_gb300 import paged
from test_gpu_paged import Case, _dev, _weigh_case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _weigh(c, nq, decay, workspace=None, max_ctx=None):
    out, w = torch.full_like(c.q, 7.0), c.w.clone()
    paged.decode_weigh(c.pool, c.q, _dev(c.tables), _dev(c.ctx), int(c.ctx.max()) if max_ctx is None else max_ctx, w,
                       _dev(c.wtables), decay, out, workspace)
    torch.cuda.synchronize()
    return out, w


def _offset_workspace(need, offset):
    """A workspace of exactly `need` bytes at `offset` past a multiple of 256, and the bytes about it, which stay 0x5a."""
    arena = torch.full((need + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    at = -arena.data_ptr() % 256 + offset
    ws, rest = arena[at:at + need], torch.ones_like(arena, dtype=torch.bool)
    rest[at:at + need] = False
    assert ws.data_ptr() % 256 == offset
    return ws, lambda: bool((arena[rest] == 0x5a).all())


@pytest.mark.parametrize("kv,group,d,rows,prefix", [
    (2, 1, 128, [18], [1500]),              # one Q tile
    (1, 20, 64, [30], [3603]),              # several
    (2, 1, 128, [1, 30] * 10, [50, 900] * 10),   # groups in the workspace too
    (2, 3, 64, [2, 3], [0, 37]),            # no prefix in one pass
])
def test_shared_takes_any_workspace_at_sixteen_bytes(kv, group, d, rows, prefix):
    ctx = [p + 9 * (i % 5) for r, p in zip(rows, prefix) for i in range(r)]
    c = Case(71, kv, group, d, rows, prefix, ctx)
    need = paged.decode_shared_workspace(len(ctx), kv * group, kv, d, max(ctx) + 700, rows, prefix)
    want = c.run(max_ctx=max(ctx) + 700)
    for offset in (0, 16, 32, 48):
        ws, whole = _offset_workspace(need, offset)
        assert torch.equal(c.run(max_ctx=max(ctx) + 700, workspace=ws), want), offset
        assert whole(), offset


@pytest.mark.parametrize("kv,group,d,ctx,nq", [
    (1, 4, 128, [1300, 40, 3], 70),         # a window's common keys in one pass
    (2, 2, 64, [700, 1500], 16),
    (1, 8, 64, [9000, 30], 1),              # splits, the join beside the weights
    (1, 8, 64, [400, 17], 1),               # scores of one split in the workspace
])
def test_weigh_takes_any_workspace_at_sixteen_bytes(kv, group, d, ctx, nq):
    c = _weigh_case(72, kv, group, d, ctx, nq)
    need = paged.decode_weigh_workspace(len(ctx), nq, kv * group, kv, d, max(ctx))
    want = _weigh(c, nq, 0.5, None)
    for offset in (0, 16, 32, 48):
        ws, whole = _offset_workspace(need, offset)
        got = _weigh(c, nq, 0.5, ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), offset
        assert whole(), offset
