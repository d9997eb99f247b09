"""A decoder layer's attention from packed weights to the residual stream: projections, prompt attention, cache and
decode steps in the order in which a program calls them. Each stage is compared with its definition in 64 bits
on the stage before's own output."""

import numpy as np
import pytest
import torch

import oracle
import weight_only_bit_qgemv_b200 as woq
from weight_only_bit_qgemv_b200 import _lib, workloads
from tests import attn_ref as ref
from tests.gpu_util import FP32_TOL, max_rel, packed_from_weight

pytestmark = pytest.mark.gpu

HEADS, KV, DIM, HIDDEN, PAGE = 4, 2, 128, 256, 32


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def layer(bits):
    n = (HEADS + 2 * KV) * DIM
    qkv = packed_from_weight(workloads.weight(n, HIDDEN, seed=1, std=0.1), bits)
    out = packed_from_weight(workloads.weight(HIDDEN, HEADS * DIM, seed=2), bits)
    return qkv, out


def heads_of(rows):
    r = rows.view(-1, HEADS + 2 * KV, DIM)
    return r[:, :HEADS], r[:, HEADS:HEADS + KV], r[:, HEADS + KV:]


def check_rows(got, q, k, v):
    """One token's attention against its definition, q [heads, dim] over k, v [tokens, kv_heads, dim] (float64)."""
    want, size = ref.attend(q, k, v, DIM**-0.5)
    err = np.abs(got - want)
    assert (err <= ref.tolerance(want, size, torch.float32)).all(), err.max()


@pytest.mark.parametrize("bits", [4, 8])
def test_prompts_then_decode_steps(bits):
    (wqkv, pk, sk), (wout, po, so) = layer(bits)
    lens = [45, 1, 130]
    batch, total = len(lens), sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    width = 8
    table = np.random.default_rng(3).permutation(batch * width).reshape(batch, width)
    cache = woq.KV4Cache.empty(batch * width, KV, DIM, PAGE)
    x = workloads.activations(total, HIDDEN, seed=4).cuda()
    table_d, cu_d = ints(table), ints(cu)

    # ---- prompts ----
    qkv = woq.qgemm(x, wqkv, path="fp32")
    assert max_rel(qkv.cpu().numpy(), oracle.qgemv_ref(x.cpu().numpy(), pk, sk, bits)) <= FP32_TOL
    q, k, v = heads_of(qkv)  # slices of the projection's rows
    woq.kv4_append(cache, k, v, cu_d, table_d)
    att = woq.attn_prompt(q, k, v, cu_d)
    q64, k64, v64 = (t.double().cpu().numpy() for t in (q, k, v))
    for b in range(batch):
        for i in {0, lens[b] // 2, lens[b] - 1}:
            at = cu[b] + i
            check_rows(att[at].double().cpu().numpy(), q64[at], k64[cu[b]:at + 1], v64[cu[b]:at + 1])
    h = woq.qgemm(att.view(total, -1), wout, path="fp32")
    assert max_rel(h.cpu().numpy(), oracle.qgemv_ref(att.view(total, -1).cpu().numpy(), po, so, bits)) <= FP32_TOL

    # ---- decode steps: as calls, then the same steps as a graph that follows the lengths on the device ----
    step_x = torch.zeros(batch, HIDDEN, device="cuda")
    qkv1 = torch.empty(batch, (HEADS + 2 * KV) * DIM, device="cuda")
    att1, hidden = torch.empty(batch, HEADS, DIM, device="cuda"), torch.empty(batch, HIDDEN, device="cuda")
    before, after, one_each = ints(lens), ints(lens) + 1, ints(range(batch + 1))
    q1, k1, v1 = heads_of(qkv1)
    ws = woq.kv4_attn_workspace(cache, q1)

    def step():
        woq.qgemv(step_x, wqkv, out=qkv1)
        woq.kv4_append(cache, k1, v1, one_each, table_d, start=before)
        woq.kv4_attn(q1, cache, after, table_d, out=att1, workspace=ws)
        hidden.copy_(step_x)
        woq.qgemv_residual(att1.view(batch, -1), wout, hidden, out=hidden)
        before.add_(1)
        after.add_(1)

    graph = None
    for n in range(6):
        step_x.copy_(workloads.activations(batch, HIDDEN, seed=10 + n))
        if n < 3:
            step()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                torch.cuda.synchronize()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        kc, vc = ref.read_pages(cache.codes, cache.scales)
        got = att1.double().cpu().numpy()
        for b in range(batch):
            count = lens[b] + n + 1
            at = [(table[b][j // PAGE], j % PAGE) for j in range(count)]
            kb, vb = (np.array([t[p, :, s] for p, s in at]) for t in (kc, vc))
            check_rows(got[b], q1[b].double().cpu().numpy(), kb, vb)
            # the newest token is this step's, as its quantiser makes it
            values = ref.quantised(k1[b].cpu().numpy())[2]
            assert np.array_equal(kb[-1], values)
        want = oracle.qgemv_ref(att1.view(batch, -1).cpu().numpy(), po, so, bits) + step_x.cpu().numpy()
        assert max_rel(hidden.cpu().numpy(), want) <= FP32_TOL
    assert before.tolist() == [n + 6 for n in lens]
    assert woq.device_status() == _lib.WOQ_OK
