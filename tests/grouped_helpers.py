"""Plumbing of the grouped-layer tests: random experts, group offsets, the
oracle's operands in the grouped scale layout, and the oracle's product."""
import numpy as np
import torch

import nvfp4_w4a4_quantized_10_b200 as nv
import oracle

I32 = torch.int32


def offsets_of(rows):
    return torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=I32)


def experts(E, N, K, seed):
    """Quantized weights of E experts: device codes, scales, global scales, and the oracle's operands."""
    r = np.random.default_rng(seed)
    codes, tc, gs, host = [], [], [], []
    for e in range(E):
        w = (r.standard_normal((N, K)) * 0.02 * (1 + e % 3)).astype(np.float32)
        g = oracle.global_scale(oracle.amax(w))
        c, s = oracle.quantize(w, g)
        codes.append(c)
        tc.append(oracle.scales_to_tc(s, K))
        gs.append(g)
        host.append((c, s, g))
    return (torch.from_numpy(np.stack(codes)).cuda(), torch.from_numpy(np.stack(tc)).cuda(),
            torch.tensor(np.array(gs, dtype=np.float32)).cuda(), host)


def grouped_scales(per_group, T, K):
    """Row-major scales of each group -> the grouped layout (other bytes 0xFF: E4M3 NaN, where nothing may be read),
    and the mask of bytes that belong to a group's rows (padding columns included)."""
    E = len(per_group)
    buf = np.full(nv.nvfp4_grouped_scale_bytes(T, E, K), 255, dtype=np.uint8)
    mask = np.zeros(buf.size, dtype=bool)
    at = 0
    for s in per_group:
        if s.shape[0] == 0:
            continue
        tc = oracle.scales_to_tc(s, K)
        used = oracle.scales_to_tc(np.ones_like(s), K).astype(bool)
        rows = np.arange(s.shape[0])
        for j in range(s.shape[1], -(-K // 64) * 4):            # padding columns of real rows
            used[((rows >> 7) * -(-K // 64) + (j >> 2)) * 512 + (rows & 31) * 16 + ((rows >> 5) & 3) * 4 + (j & 3)] = True
        buf[at:at + tc.size][used] = tc[used]
        mask[at:at + tc.size] = used
        at += tc.size
    return buf, mask


def activation(T, K, seed):
    r = np.random.default_rng(seed)
    x = r.standard_normal((T, K)).astype(np.float32)
    x[:, r.integers(0, K, max(1, K // 500))] *= 40.0
    return x


def oracle_rows(x, rows, gs, T, K):
    """Quantize each group's rows of x with its own scale: codes [T, K/2] (rows past the groups 0xFF), per-group scales."""
    codes = np.full((T, K // 2), 255, dtype=np.uint8)
    per, at = [], 0
    for n, g in zip(rows, gs):
        if n:
            c, s = oracle.quantize(np.ascontiguousarray(x[at:at + n]), np.float32(g))
            codes[at:at + n] = c
        else:
            s = np.zeros((0, K // 16), dtype=np.uint8)
        per.append(s)
        at += n
    return codes, per


def product(codes, per, ga, host, rows, N):
    """Oracle (FP64) product of every group; rows past the groups are absent."""
    out, at = [], 0
    for e, n in enumerate(rows):
        if n:
            wc, ws, gw = host[e]
            out.append(oracle.gemm(np.ascontiguousarray(codes[at:at + n]), per[e], np.float32(ga[e]), wc, ws, gw))
        at += n
    return np.concatenate(out) if out else np.zeros((0, N))
