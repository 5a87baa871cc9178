"""What the key/value cache's entry points write, on the GPU: every element that they owe, in both types and with
rows that are whole, cut, empty and NaN; and no byte outside their outputs and the workspace they asked for."""
import numpy as np
import pytest
import torch

import block_scaled_precision_mx_gb300 as mx
from tests.test_gpu_kv import attention_case, built, check_attention, gpu, values  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,elem", [("bf16", 0), ("f16", 0), ("f16", 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("queries", [3, 9, 30, 100, 300])
def test_whole_cut_empty_and_nan_rows_in_both_types(queries, d, kind, elem):
    """Long contexts whose work several CTAs share, short ones that one has, queries without tokens, and NaN in a
    value that half of the rows see."""
    rng = np.random.RandomState(queries + d)
    lens, q = [6000, 40, 0, 2500, 129], [queries, min(queries, 50), 2, queries, 129]
    c = attention_case(rng, lens, q, 4, 2, d, 64, kind, elem, q_pad=5)
    for r in (0, 3):
        at = lens[r] - queries // 2 - 1
        c["vc"][c["tables"][r, at // 64], 1, at % 64, 5] = 0x7F
        c["vc"][c["tables"][r, 1], 0, 3, d - 1] = 0x7F
    check_attention(c, elem)


# ------------------------------------------------------------------ guard bands
FILL, GUARD = 0xA5, 4096


class Guarded:
    """A tensor of this shape and type between two guard bands of FILL bytes; holds FILL itself, or `like`."""

    def __init__(self, shape, dtype, like=None):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((2 * GUARD + n,), FILL, dtype=torch.uint8, device="cuda")
        self.t = self.raw[GUARD:GUARD + n].view(dtype).view(*shape)
        if like is not None:
            self.t.copy_(like)

    def intact(self):
        return bool((self.raw[:GUARD] == FILL).all()) and bool((self.raw[GUARD + self.t.numel() * self.t.element_size():] == FILL).all())


def check(bufs, what):
    torch.cuda.synchronize()
    assert mx.mx_check() == mx.MX_OK, what
    bad = [n for n, b in bufs.items() if not b.intact()]
    assert not bad, f"{what}: a guard band of {bad} was written"


@pytest.mark.parametrize("before,after,p,tokens", [
    ([0], [1], 16, 1), ([5, 0, 90], [6, 33, 0], 16, 40), ([0, 128, 7], [300, 129, 8], 128, 305),
    ([3] * 700, [4] * 700, 64, 701), ([0, 50], [2000, 0], 32, 2000)])
def test_block_tables_write_only_their_outputs(before, after, p, tokens):
    before, after = np.array(before), np.array(after)
    held, want = -(-before // p), -(-after // p)
    width, blocks = int(max(held.max(), want.max())), int(held.sum() + np.maximum(want - held, 0).sum())
    tables, order = np.full((len(before), width), -1), np.random.RandomState(p).permutation(blocks)
    at = np.concatenate([[0], np.cumsum(held)])
    for r, h in enumerate(held):
        tables[r, :h] = order[at[r]:at[r + 1]]
    i32, i64 = torch.int32, torch.int64
    b = {"tables": Guarded(tables.shape, i32, gpu(tables)), "free": Guarded((blocks,), i32, gpu(np.roll(order, -at[-1]))),
         "q_start": Guarded((len(before) + 1,), i32), "slots": Guarded((tokens,), i64),
         "positions": Guarded((tokens,), i32), "info": Guarded((2,), i32)}
    count = torch.tensor([blocks - at[-1]], dtype=i32, device="cuda")
    mx.kv_block_tables(b["tables"].t, gpu(before, i32), gpu(after, i32), b["free"].t, count, tokens, p,
                       b["q_start"].t, b["slots"].t, b["positions"].t, b["info"].t)
    check(b, f"kv_block_tables {len(before)} requests")
    new = int(np.maximum(after - before, 0).sum())
    assert (b["slots"].t[:new] >= 0).all() and (b["slots"].t[new:] == -1).all() and b["q_start"].t[-1] == new


@pytest.mark.parametrize("d,p,h", [(64, 16, 1), (128, 16, 3), (64, 128, 2), (128, 64, 5), (128, 128, 1)])
@pytest.mark.parametrize("tokens", [1, 37, 300])
def test_append_writes_only_the_cache(d, p, h, tokens):
    rng = np.random.RandomState(tokens)
    blocks = -(-(tokens + 3) // p)
    b = {"k": Guarded((blocks, h, p, d), torch.uint8), "v": Guarded((blocks, h, p, d), torch.uint8),
         "k_scale": Guarded((blocks, h), torch.float32, torch.ones(blocks, h)),
         "v_scale": Guarded((blocks, h), torch.float32, torch.ones(blocks, h))}
    slots = np.arange(3, 3 + tokens)                              # from a first block in use to the last block
    x = values(rng, (tokens, h, d), torch.float16).cuda()
    mx.kv_cache_append(x, x, gpu(slots), b["k"].t, b["v"].t, b["k_scale"].t, b["v_scale"].t)
    check(b, f"kv_cache_append {tokens} tokens")
    rows = b["k"].t.transpose(1, 2).reshape(blocks * p, h, d)      # token by token
    assert (rows[3 + tokens:] == FILL).all() and not (rows[3:3 + tokens] == FILL).all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("lens,queries,heads,kv_heads", [
    ([1], [1], 1, 1), ([70, 0, 9000], [1, 1, 1], 8, 2), ([70, 5, 3000], [4, 5, 3], 6, 2), ([90, 4000], [17, 50], 4, 4),
    ([300], [300], 8, 1), ([100] * 520 + [3000], [17] * 521, 2, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_writes_only_its_outputs_and_its_workspace(d, lens, queries, heads, kv_heads, kind):
    c = attention_case(np.random.RandomState(d), lens, queries, heads, kv_heads, d, 16, kind, 0, q_pad=3)
    args = [c["q"], *(gpu(c[n]) for n in ("kc", "vc", "ks", "vs", "tables", "lens", "q_start"))]
    t, most = len(c["q"]), max(queries)
    need = mx.kv_attention_workspace_bytes(t, len(lens), most, heads, kv_heads, d)
    b = {"out": Guarded((t, heads, d), c["q"].dtype), "lse": Guarded((t, heads), torch.float32),
         "workspace": Guarded((need,), torch.uint8)}
    b["workspace"].t[:4096] = 0
    for _ in range(2):
        mx.kv_attention(*args, most, out=b["out"].t, lse=b["lse"].t, workspace=b["workspace"].t)
        check(b, f"kv_attention {queries[:3]} queries")
    assert not b["workspace"].t[:4096].any()
    want = mx.kv_attention(*args, most)
    assert torch.equal(b["out"].t, want[0]) and torch.equal(b["lse"].t, want[1])
