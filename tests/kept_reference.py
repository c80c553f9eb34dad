"""Plain numpy forms of rows in 8 bits and of SwiGLU, written from their definitions."""
import numpy as np
import torch


def bits(t):
    """uint16 bits of a bf16 tensor."""
    return t.contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def bf16(b):
    """The bf16 tensor of uint16 bits."""
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).view(torch.bfloat16)


def keep(x):
    """(codes int8, exponents uint8) of a bf16 tensor [rows, width], value by value."""
    b = bits(x)
    rows, width = b.shape
    groups = -(-width // 32)
    exponents = np.zeros((rows, groups), np.uint8)
    codes = np.zeros((rows, width), np.int8)
    values = x.cpu().double().numpy()
    for g in range(groups):
        part = slice(32 * g, min(width, 32 * g + 32))
        e = ((b[:, part] >> 7) & 255).max(1)
        exponents[:, g] = e
        fine = e < 255
        # np.ldexp is exact; np.round goes half to even
        q = np.round(np.ldexp(values[fine, part], (133 - e[fine].astype(np.int64))[:, None]))
        codes[fine, part] = np.clip(q, -127, 127).astype(np.int8)
    return torch.from_numpy(codes), torch.from_numpy(exponents)


def restore(codes, exponents):
    """What the codes stand for, bf16 (exactly)."""
    e = np.repeat(exponents.cpu().numpy().astype(np.int64), 32, axis=1)[:, :codes.shape[1]]
    v = np.ldexp(codes.cpu().numpy().astype(np.float64), e - 133)
    v[e == 255] = np.nan
    t = torch.from_numpy(v).to(torch.bfloat16)
    assert np.array_equal(np.nan_to_num(t.double().numpy()), np.nan_to_num(v))
    return t


def swiglu(gu):
    """h in float64 from float64 rows [g, u]."""
    g, u = gu.chunk(2, dim=1)
    return g * torch.sigmoid(g) * u


def swiglu_backward(dh, gu):
    """dgu in float64; 1 - s is the sigmoid of -g."""
    g, u = gu.chunk(2, dim=1)
    s = torch.sigmoid(g)
    return torch.cat([dh * u * s * (1 + g * torch.sigmoid(-g)), dh * g * s], dim=1)
