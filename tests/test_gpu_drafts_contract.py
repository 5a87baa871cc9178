"""Drafted tokens at the ends of what their entry points document, on the GPU against the 64-bit reference."""
import numpy as np
import pytest
import torch

from tests.test_gpu_drafts import check_verify

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


# ------------------------------------------------------------------ verification
STARS = {  # the root's target and draft rows, and tokens that its children take in turn
    "half": ([1 / 2, 1 / 2], [1, 0], [0]), "quarter": ([1 / 4, 3 / 4], [1, 0], [0]), "sixteenth": ([1 / 16, 15 / 16], [1, 0], [0]),
    "two": ([1 / 4, 1 / 4, 1 / 2], [1 / 2, 1 / 2, 0], [0, 1, 1]), "apart": ([1 / 4, 1 / 4, 1 / 2, 0, 0], [1 / 2, 0, 0, 1 / 4, 1 / 4], [3, 0, 4]),
    "most": ([1 / 8, 1 / 8, 3 / 4], [3 / 4, 1 / 4, 0], [0, 1, 0, 0])}


@pytest.mark.parametrize("below", [0, 1])
@pytest.mark.parametrize("children", [17, 18, 22, 31, 32, 33, 63, 64, 65, 200, 1022])
@pytest.mark.parametrize("star", list(STARS))
def test_verify_siblings_of_a_narrow_draft(star, children, below):
    """One node's many children, drawn from few tokens, so that W q passes 16, 32 and more: what is used up stays so.  Rows and
    random numbers are dyadic, so that the reference's sums and products are exact, and it is exact what the next token is."""
    p, q, turns = STARS[star]
    n = 1 + below + children  # (below: the parent is a child of the root, which is accepted)
    parents = np.int32([-1] + [0] * below + [below] * children)
    drafts = np.int32([-7] + [len(p) - 1] * below + [turns[i % len(turns)] for i in range(children)])
    target, draft = np.tile(np.float32(p), (n, 1)), np.tile(np.float32(q), (n, 1))
    if below:
        target[0] = draft[0] = np.eye(len(p))[len(p) - 1]
    rng = np.random.RandomState(children)
    for trial in range(4):
        accept = (rng.randint(1 << 9, 1 << 10, n) / 1024).astype(np.float32)  # 1/2 and above: rejected by all of the rows
        if trial:  # behind the first few, which use their tokens up, any number
            accept[below + 5:] = (rng.randint(0, 1 << 10, n - below - 5) / (1024 << 4 * trial)).astype(np.float32)
        if star == "half":
            accept[1 + below] = 0.5 if trial else accept[1 + below]
        if below:
            accept[1] = 0.25
        for sample in (0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24):
            want = check_verify([n], len(p), False, target=target, draft=draft, drafts=drafts, parents=parents, accept=accept,
                                sample=np.float32([sample]))
            if trial == 0:
                assert int(want[2][0]) == 1 + below  # (a word on the inputs: all of them are rejected)
