"""A step's metadata from request lengths, one request and one token at a time.

TEST INFRASTRUCTURE (see the package docstring). Plain Python integers; the rule
is the one the header states for msa_build_step.
"""
from __future__ import annotations

import numpy as np

BAD_PAGE, BAD_SEQLEN, NO_PAGES = 0x1, 0x4, 0x40


def build_step(ctx, new, free_pages, free_head, table, num_pages, max_tokens, axes=1, pos_offset=None, block=128):
    """Returns dict(table, seq_lens, token_starts, slots, positions, free_head, flags)."""
    table = np.array(table, dtype=np.int64)
    B, NB = table.shape
    cap = NB * block
    out = dict(seq_lens=[], token_starts=[], slots=[-1] * max_tokens, positions=[0] * max_tokens, flags=0)
    head, taken, at = int(free_head), 0, 0
    cursor = head
    for b in range(B):
        c, n = int(ctx[b]), int(new[b])
        add = max(n, 0)
        ok = c >= 0 and n >= 0 and c + n <= cap
        first_blk, need = -(-c // block), 0
        if ok:
            need = -(-(c + n) // block) - first_blk
        placed = ok and at + add <= max_tokens
        fits = need == 0 or (head >= 0 and cursor + need <= len(free_pages))
        out["token_starts"].append(min(at, max_tokens))
        if not placed:
            out["flags"] |= BAD_SEQLEN
        elif not fits:
            out["flags"] |= NO_PAGES
        if placed and fits:
            for i in range(need):
                page = int(free_pages[cursor + i])
                if not 0 <= page < num_pages:
                    out["flags"] |= BAD_PAGE
                    page = -1
                table[b, first_blk + i] = page
            taken += need
        out["seq_lens"].append(c + add if placed and fits else min(max(c, 0), cap))
        for i in range(add):
            t = at + i
            if t >= max_tokens:
                break
            p = c + i
            out["positions"][t] = p + (0 if pos_offset is None else int(pos_offset[b]))
            if placed and fits:
                page = int(table[b, p // block])
                if 0 <= page < num_pages:
                    out["slots"][t] = page * block + p % block
                else:
                    out["flags"] |= BAD_PAGE
        at += add
        cursor += need
    out["token_starts"].append(min(at, max_tokens))
    out["free_head"] = head + taken
    out["positions"] = np.tile(np.array(out["positions"], dtype=np.int64).astype(np.int32), (axes, 1))   # wraps, as int32 does
    out["slots"] = np.array(out["slots"], dtype=np.int64)
    out["seq_lens"] = np.array(out["seq_lens"], dtype=np.int32)
    out["token_starts"] = np.array(out["token_starts"], dtype=np.int32)
    out["table"] = table.astype(np.int32)
    return out
