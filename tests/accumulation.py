"""How far sums in fp32 may be off, by the way they are added up.

u = 2^-24, half a step of fp32.  A sum's terms t have zero mean, q = sqrt(sum t^2):
after a share s of them the partial sum has size q sqrt(s).

Largest error: every addition on the longest way of a term is off by at most 2 u
of the sum of magnitudes (a matrix instruction may cut rather than round).
Root mean square over many sums:
  cut (always towards zero, by u of the partial sum on average): the errors of L
  additions in a row have the signs of slowly changing partial sums and add up to
  u q L / sqrt(3);
  rounded (any sign, u / sqrt(3) of it): to u q sqrt(L) / 2, less than u q sqrt(L).
"""
import numpy as np

U = 2.0 ** -24
INNER = 32                               # products that one matrix instruction adds


def product_chain(T, K):
    """(additions into one accumulator, further ones) on the longest way of a term
    of a product with 4-bit weights.  Up to two tokens: 512 columns a wave and up to
    eight waves, 32 products a lane of each, then four lanes' sums and the waves'.
    More: chunks of 128 columns, one wave up to four of them, two up to eight, at
    least four beyond; each instruction adds 32 products."""
    if T <= 2:
        groups = -(-K // 512)
        waves = min(8, groups)
        return 32 * -(-groups // waves), 4 + waves + 1
    chunks = -(-K // 128)
    waves = 1 if chunks <= 4 else 2 if chunks <= 8 else 4
    return 4 * -(-chunks // waves), INNER + 8 + 1


def product_error(got, x, w, T, K):
    """(largest error, root mean square) of products in units of what they may be."""
    ref, mag, q = x @ w.T, np.abs(x) @ np.abs(w).T, np.sqrt((x * x) @ (w * w).T)
    long, more = product_chain(T, K)
    err = np.abs(got - ref)
    return (err / ((2 * (long + more) + 2) * U * mag)).max(), np.sqrt(((err / (U * q)) ** 2).mean()) / ((long + more) / np.sqrt(3) + 2)


def column_chain(T, parts):
    """Additions on the longest way of a row into a column's sum: the rows of a part
    over the up to 16 that its workgroup takes at once, those 16, and the parts, 32 in
    turn.  (Up to 1024 rows at least 64 threads take the rows: 16 each, five steps over
    lanes and up to 16 waves, which is less.)"""
    return -(-T // parts) + 16 + -(-parts // 32) + 32


def column_error(got, terms, T, parts):
    """The same of column sums of rounded terms (two roundings each)."""
    ref, mag, q = terms.sum(axis=0), np.abs(terms).sum(axis=0), np.sqrt((terms * terms).sum(axis=0))
    n = column_chain(T, parts)
    err = np.abs(got - ref)
    return (err / ((n + 2) * U * mag)).max(), np.sqrt(((err / (U * q)) ** 2).mean()) / (np.sqrt(n) + 2)
