"""A bound on 8-bit decode attention that holds its weights to 20 bits, for scores of a few units,
where many positions carry weight."""
import numpy as np


def attend_and_bound(q, k, v, exact_scores):
    """softmax(q k^T) v in 64 bits and a bound on a kernel's error, both [G, D].

    To first order the output moves by the sum of w_i d_i (v_i - o), d_i a weight's relative error:
      2^-20: 2^x is good to 2^-22, the two halves of a weight hold 22 bits, and the exponent,
             a difference below 16 in magnitude for weights that count, is rounded by at most
             2^-21, which is ln(2) of that in the weight;
      the score's error, exact_scores: |s| 2^-23, for the rounded log2(e) and one product; else
             40 roundings of the sum of |q| |k|, as in attend_tolerance.
    Numerator and normaliser are sums of two or more chains of blocks, with at most 8 roundings
    within a block and where the chains join, each up to 2^-24 of the sum of w |v|."""
    s = q @ k.T
    w = np.exp(s - s.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    o = w @ v
    d = 2.0 ** -20 + (np.abs(s) * 2.0 ** -23 if exact_scores
                      else 40 * 2.0 ** -24 * (np.abs(q) @ np.abs(k).T))
    chain = (k.shape[0] + 15) // 16 / 2 + 8
    bound = np.empty_like(o)
    for g in range(q.shape[0]):
        bound[g] = (w[g] * d[g]) @ np.abs(v - o[g]) + 2 * chain * 2.0 ** -24 * (w[g] @ np.abs(v))
    return o, bound
