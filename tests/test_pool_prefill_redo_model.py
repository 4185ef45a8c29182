"""A model of one softmax warp of the pool pre-fill kernel (prefill_pool_kernel) and its
tensor-memory stores, which are asynchronous: they land one by one, in any order, until a
wait for all of them.  A tile whose largest logit passes the reference m by more than 2^8
stores its first three blocks of weights, rescales O, and stores them again relative to the
new m; the product that follows has to read the second ones.  Scheduler and checks are
those of tests/protocol_sim.py.  On the GPU: logits that move the reference in every tile."""
import numpy as np
import pytest
import torch

import oracle
from head_split_kv_duo_b200 import inputs
from parity import bits
from protocol_sim import Sim, wait
from test_pool_prefill import DEV, Tokens, _gpu_pool

EARLY, BLOCKS, OPARTS = 3, 4, 2  # blocks of weights handed over first, all blocks; parts of O


def warp(sim, redone, wait_between=True, wait_before_rest=True):
    """`redone`: per tile, whether its reference moves.  The keyword arguments plant mistakes."""
    for name in ("SFull", "PFull", "PRest"):
        sim.bar(name)
    flying = [0]

    def lands(buf, version):
        yield None
        sim.write(buf, version)
        flying[0] -= 1

    def store(buf, version):
        flying[0] += 1
        sim.spawn(lands(buf, version), f"store {buf}")

    def all_landed():
        while flying[0]:
            yield None

    def softmax():
        ref = 0  # changes of the reference so far
        for j, redo in enumerate(redone):
            yield wait("SFull", j)
            for b in range(EARLY):
                store(f"p{b}", (j, ref))
                yield None
            if redo:
                ref += 1
                if wait_between:
                    yield from all_landed()
                for b in range(OPARTS):
                    if j > 0:
                        sim.read(f"o{b}", ("product", j - 1))
                    store(f"o{b}", ("rescaled", j, ref))
                    yield None
                for b in range(EARLY):
                    store(f"p{b}", (j, ref))
                    yield None
            yield from all_landed()
            sim.arrive("PFull")
            for b in range(EARLY, BLOCKS):
                store(f"p{b}", (j, ref))
            if wait_before_rest:
                yield from all_landed()
            sim.arrive("PRest")

    def products():
        ref = 0
        for j, redo in enumerate(redone):
            sim.arrive("SFull")
            ref += redo
            for name, blocks in (("PFull", range(EARLY)), ("PRest", range(EARLY, BLOCKS))):
                yield wait(name, j)
                for b in blocks:
                    sim.read(f"p{b}", (j, ref))
                    yield None
            for b in range(OPARTS):
                if redo:
                    sim.read(f"o{b}", ("rescaled", j, ref))
                sim.write(f"o{b}", ("product", j))

    sim.spawn(softmax(), "softmax")
    sim.spawn(products(), "products")


TILES = [[0], [1], [0, 1], [1, 1, 1], [0, 1, 0, 0, 1, 1], [1] * 8, [0] * 8]


@pytest.mark.parametrize("redone", TILES, ids=str)
def test_redone_weights_are_what_the_product_reads(redone):
    for seed in range(300):
        sim = Sim(seed)
        warp(sim, redone)
        sim.run()


@pytest.mark.parametrize("mistake", ["wait_between", "wait_before_rest"])
def test_model_catches(mistake):
    caught = 0
    for seed in range(300):
        sim = Sim(seed)
        warp(sim, [0, 1, 1, 0, 1], **{mistake: False})
        try:
            sim.run()
        except AssertionError:
            caught += 1
    assert caught > 0


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,mask,S,W", [(8, [1, 0], 4, 300), (2, [1, 0], 130, 700), (16, [1], 0, 64)])
def test_references_that_move_in_every_tile(Hq, mask, S, W):
    """Logits that grow by 8 (11.5 in base 2, past the slack of 8) from a tile to the next, four
    times over, in pages, rings and the call's own rows, against the oracle.  128 products of
    0.25 and 0.25 times a factor of at most 15.25 are a sum |q k| of 122, and with scale 0.2 a
    logit of 25, off by at most 128 * 2^-24 * 25 < 2^-12.

    Only bounds relative to each element are asked.  Outputs here reach 0.25 * 15.25 = 3.8, and
    from 2 to 4 bf16 values are 2^-6 apart: the result's own rounding, uniform over half a
    step, is 2^-8 = 3.9e-3 on average, more than the mean error of 2e-3 that holds for
    outputs below one."""
    tk = Tokens(_gpu_pool(Hq, len(mask), mask, S, W, softmax_scale=0.2), 11000)
    tk.draw = lambda n, heads: _rising(tk, n, heads)
    tk.check = lambda *args: _bounded(tk, *args)
    seqs = [tk.open(x) for x in (0, 700, 1500)]
    tk.prefill(0, seqs, [900, 129, 33], rows=60, scale=0.2)
    tk.prefill(0, seqs[::-1], [1, 300, 77], rows=60, scale=0.2)
    tk.check_cache()
    assert tk.pool.device_status() == 0


def _bounded(tk, layer, q, k, v, pos0, out, lse, pick, scale, what):
    """Weights and result rounded to bf16, half a step (2^-8) each; logits off by 2^-12; the sum of
    weights, over at most 15 tiles of 128 in 32 bits, by less than 5e-5."""
    pool, Hq = tk.pool, q.shape[1]
    rows = None if pick is None else [r * Hq + h for r in pick for h in range(Hq)]
    args = (pool.mask[layer].numpy().astype(bool), pool.S, pool.W)
    w, wl = oracle.attend(bits(q[None]), bits(k[None]), bits(v[None]), *args, pos0=pos0, scale=scale, rows=rows)
    size, _ = oracle.attend(bits(q[None]), bits(k[None]), bits(v[None].abs()), *args, pos0=pos0, scale=scale,
                            rows=rows)
    o, l = (x.float().cpu().numpy() if pick is None else x.float().cpu().numpy()[pick] for x in (out, lse))
    w, size, wl = (x.reshape(y.shape) for x, y in ((w, o), (size, o), (wl, l)))
    off = np.abs(o - w) / (2.0 ** -8 * np.abs(w) + (2.0 ** -8 + 2.0 ** -12) * size)
    assert off.max() <= 1, f"{what}: {off.max()} of the tolerance"
    assert np.abs(l - wl).max() <= 2.0 ** -12 + 5e-5, f"{what}: lse off by {np.abs(l - wl).max()}"


def _rising(tk, n, heads):
    """Rows around 0.25; keys and values times 5 a tile."""
    tk.seed += 1
    x = 0.01 * inputs.randn((n, heads, 128), tk.seed, device=DEV).float() + 0.25
    if heads == tk.pool.kv_heads:
        x *= (0.25 + 5 * (torch.arange(n, device=DEV) // 128 % 4))[:, None, None]
    return x.to(torch.bfloat16)
