"""Plain 64-bit implementations of the dense path in 8 bits, for its tests."""
import math

import torch

MAGNITUDES = torch.tensor([(c % 8) / 512 if c < 8 else (1 + (c % 8) / 8) * 2.0 ** (c // 8 - 7) for c in range(127)],
                          dtype=torch.float64)
BORDERS = (MAGNITUDES[1:] + MAGNITUDES[:-1]) / 2


def e4m3_codes(q):
    """Codes (0 .. 255) of 64-bit values, to nearest even, at most 448."""
    size = q.abs()
    b = BORDERS.to(q.device)
    code = torch.bucketize(size, b)
    tie = (code < 126) & (size == b[code.clamp(max=125)])
    code = code + (tie & (code % 2 == 1))
    return torch.where(torch.signbit(q), code + 128, code)


def quantize(v):
    """v [rows, d] in 64 bits: codes (int64), scales (float32 values)."""
    rows, d = v.shape
    nb = -(-d // 128)
    p = torch.zeros(rows, nb * 128, dtype=torch.float64, device=v.device)
    p[:, :d] = v
    p = p.view(rows, nb, 128)
    scales = (p.abs().amax(-1) / 448).float()
    s = scales.double()[..., None]
    q = torch.where(s > 0, p / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(p)).clamp(-448, 448)
    return e4m3_codes(q).view(rows, -1)[:, :d], scales


def values(codes, scales):
    """What codes (float8_e4m3fn) and scales [rows, blocks] stand for, in 64 bits."""
    k = codes.shape[-1]
    return codes.double() * scales.double().repeat_interleave(128, -1)[..., :k]


def weight_values(codes, scales):
    n, k = codes.shape[-2:]
    s = scales.double().repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]
    return codes.double() * s


def rms_norm(h, weight, eps, one_plus):
    w = weight.double() + (1.0 if one_plus else 0.0)
    return h.double() / torch.sqrt(h.double().square().mean(-1, keepdim=True) + eps) * w


def logprobs(logits, tokens, top, scale):
    """(logprobs, lse, entropy, ids, their logprobs, sum p |x - max|) of a row at a time."""
    out = []
    for row, toks in zip(logits.double().cpu(), tokens.cpu().tolist()):
        x = row * scale
        v = len(row)
        if torch.isnan(x).any() or (x == math.inf).any():
            lse = ent = math.nan
            lp = torch.full((v,), math.nan, dtype=torch.float64)
            spread = 0.0
        elif (x == -math.inf).all():
            lse, ent, spread = -math.inf, 0.0, 0.0
            lp = torch.full((v,), -math.inf, dtype=torch.float64)
        else:
            most = x.max()  # taken off first: next to values of the type's lowest, a log of the sum would be lost
            logs = float(torch.log(torch.exp(x - most).sum()))
            lse = float(most) + logs
            lp = (x - most) - logs
            p = lp.exp()
            live = p > 0
            ent = float(-(p[live] * lp[live]).sum())
            spread = float((p[live] * (x.max() - x[live])).sum())
        given = [float(lp[t]) if 0 <= t < v else (math.nan if math.isnan(lse) else -math.inf) for t in toks]
        order = torch.where(torch.isnan(row), torch.full_like(row, -math.inf), row) + 0.0
        ids = sorted(range(v), key=lambda i: (-float(order[i]), i))[:top] if top else []
        tops = [math.nan if math.isnan(lse) else float(lp[i]) for i in ids]
        out.append((given, lse, ent, ids, tops, spread))
    return out
