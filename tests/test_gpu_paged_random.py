"""The paged cache's operators over seeded random shapes, on the GPU against the
definitions in 64 bits: query heads per kv head that do and do not divide a
tile of rows, prompts of several row tiles beside single tokens and empty
sequences, trees, pages, layouts, both types."""
import os

import numpy as np
import pytest
import torch

from paged_reference import path_to
from speculative_decoding_verification_24_gb300 import rope_inv_freq, spec_kv_commit
from speculative_decoding_verification_24_gb300.build import build
from test_gpu_kv_cache import Batch, commit_reference
from test_gpu_paged_attention import BF16, FP16, Case, random_tree

pytestmark = pytest.mark.gpu

# SV_SOAK_CASES raises the counts (a longer soak of the same seeded cases)
N_CASES = int(os.environ.get("SV_SOAK_CASES", "24"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def draw_heads(rng):
    G = int(rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16]))
    Hkv = int(rng.integers(1, 5)) if G <= 8 else int(rng.integers(1, 3))
    return G * Hkv, Hkv


def draw_common(rng):
    return dict(D=int(rng.choice([64, 128])), page=int(rng.choice([8, 16, 24, 32, 48, 64, 128, 256])),
                dtype=BF16 if rng.random() < 0.5 else FP16, layout=str(rng.choice(["tokens", "heads", "halves"])))


@pytest.mark.parametrize("i", range(N_CASES))
def test_attention(i):
    rng = np.random.default_rng(3000 + i)
    Hq, Hkv = draw_heads(rng)
    kind = str(rng.choice(["prompts", "prompts", "drafts", "trees", "mixed"]))
    parents = None
    if kind == "prompts":
        # several pairs of row tiles: 128 // G tokens a tile, 2 tiles a pair
        tile = 128 // (Hq // Hkv)
        seqs = [(int(rng.choice([0, rng.integers(0, 300), rng.integers(300, 1500)])), int(rng.integers(1, 9 * tile)) % 600 + 1)
                for _ in range(int(rng.integers(1, 5)))]
    elif kind == "drafts":
        seqs = [(int(rng.integers(0, 3000)), int(rng.integers(0, 18))) for _ in range(int(rng.integers(1, 60)))]
    elif kind == "trees":
        N = int(rng.integers(1, 33))
        seqs = [(int(rng.integers(0, 700)), int(rng.integers(0, N + 1))) for _ in range(int(rng.integers(1, 20)))]
        parents = np.stack([random_tree(n, N, rng, chain=float(rng.random())) for _, n in seqs])
    else:
        seqs = [(int(rng.integers(0, 900)), int(rng.choice([0, 1, 1, 1, 5, 40, 260]))) for _ in range(int(rng.integers(2, 14)))]
    c = Case(seqs, Hq=Hq, Hkv=Hkv, parents=parents, seed=i, q_scale=float(rng.choice([0.5, 2.0, 8.0])), **draw_common(rng))
    out = c.run()
    c.check(out)
    assert torch.equal(c.run(), out)


@pytest.mark.parametrize("i", range(N_CASES))
def test_append_and_commit(i):
    rng = np.random.default_rng(5000 + i)
    Hq, Hkv = draw_heads(rng)
    common = draw_common(rng)
    tree = rng.random() < 0.6
    N = int(rng.integers(1, 33))
    count = int(rng.choice([1, rng.integers(2, 30), rng.integers(100, 400)]))
    top = N + 1 if tree or count > 30 else 60
    seqs = [(int(rng.integers(0, 200)), int(rng.integers(1 if tree else 0, max(2, min(top, 1500 // count))))) for _ in range(count)]
    parents = np.stack([random_tree(n, N, rng, chain=float(rng.random())) for _, n in seqs]) if tree else None
    if tree:
        seqs = [(c, min(n, N)) for c, n in seqs]
    b = Batch(seqs, Hq=Hq, Hkv=Hkv, seed=i, **common)
    before = b.k_cache.clone(), b.v_cache.clone()
    rotary = int(rng.choice([0, 16, 48, 64, common["D"]]))
    f, inter = (rope_inv_freq(rotary, float(rng.choice([1e4, 5e5]))) if rotary else None), bool(rng.random() < 0.5)
    dev = None if parents is None else torch.from_numpy(parents).cuda()
    positions = rng.integers(-2 ** 31, 2 ** 31, int(b.cu[-1])).astype(np.int32) if rng.random() < 0.3 else None
    q_out = b.append(q=b.q, inv_freq=f, interleaved=inter, tree_parents=dev,
                     positions=None if positions is None else torch.from_numpy(positions).cuda())
    b.check(before, b.q, q_out, f, inter, parents, positions)
    if not tree:
        return
    last = np.array([int(rng.integers(0, n)) for _, n in seqs], np.int32)
    n = np.array([len(path_to(parents[s], int(x))) - 1 for s, x in enumerate(last)], np.int32)
    n[rng.random(count) < 0.1] = -1
    k, v, lens = commit_reference(b, parents, n, last, None)
    got = spec_kv_commit(b.k_cache, b.v_cache, b.args[0], b.args[1], torch.from_numpy(n).cuda(), tree_parents=dev,
                         last_node=torch.from_numpy(last).cuda(), status_word=b.status)
    torch.cuda.synchronize()
    assert int(b.status) == 0 and np.array_equal(got.cpu().numpy(), lens)
    assert torch.equal(b.k_cache, k) and torch.equal(b.v_cache, v)
