"""Plain forms of the experts' operators, in numpy, written from their definitions
(include/okls_experts.h).  Test infrastructure: nothing on the product path uses it."""
import numpy as np


def capacity(tokens, each, n_experts, align):
    pairs = tokens * each
    return (pairs + min(pairs, n_experts) * (align - 1)) // align * align


def plan(choice, n_experts, align):
    """(rows, pairs, offsets, counts) of choice (tokens, each)."""
    tokens, each = choice.shape
    mine = [[] for _ in range(n_experts)]
    for i, e in enumerate(choice.reshape(-1).tolist()):
        if 0 <= e < n_experts:
            mine[e].append(i)
    rows = np.full(tokens * each, -1, np.int32)
    pairs = np.full(capacity(tokens, each, n_experts, align), -1, np.int32)
    offsets, counts = np.zeros(n_experts + 1, np.int32), np.array([len(m) for m in mine], np.int32)
    for e, m in enumerate(mine):
        offsets[e + 1] = offsets[e] + -(-len(m) // align) * align
        for r, i in enumerate(m):
            rows[i] = offsets[e] + r
            pairs[offsets[e] + r] = i
    return rows.reshape(tokens, each), pairs, offsets, counts


def gather(x, pairs, each):
    out = np.zeros((pairs.size, x.shape[1]))
    some = pairs >= 0
    out[some] = x[pairs[some] // each]
    return out


def combine(y, rows, weights):
    """(sums, sums of sizes)."""
    out, size = np.zeros((rows.shape[0], y.shape[1])), np.zeros((rows.shape[0], y.shape[1]))
    for t, k in zip(*np.nonzero(rows >= 0)):
        part = y[rows[t, k]] * (1.0 if weights is None else weights[t, k])
        out[t] += part
        size[t] += np.abs(part)
    return out, size


def combine_backward(dout, y, rows, pairs, weights):
    """(dy, dweights, dweights' sums of sizes)."""
    dy, dw, size = np.zeros(y.shape), np.zeros(weights.shape), np.zeros(weights.shape)
    for t, k in zip(*np.nonzero(rows >= 0)):
        r = rows[t, k]
        dy[r] = weights[t, k] * dout[t]
        dw[t, k] = dout[t] @ y[r]
        size[t, k] = np.abs(dout[t]) @ np.abs(y[r])
    return dy, dw, size


def expert_of(pairs, choice):
    """Each row's expert, -1 without a choice."""
    flat = np.append(choice.reshape(-1), -1)
    return np.where(pairs >= 0, flat[pairs], -1)


def matmul(a, b, pairs, choice):
    """(a's rows times their expert's b transposed, sums of sizes) for b (experts, n, k)."""
    out, size = np.zeros((a.shape[0], b.shape[1])), np.zeros((a.shape[0], b.shape[1]))
    of = expert_of(pairs, choice)
    for e in range(b.shape[0]):
        r = of == e
        out[r], size[r] = a[r] @ b[e].T, np.abs(a[r]) @ np.abs(b[e]).T
    return out, size


def weight_grad(a, b, pairs, choice, n_experts):
    """For each expert a's columns times b's over its rows, and the sums of sizes."""
    of = expert_of(pairs, choice)
    out = np.stack([a[:, of == e] @ b[:, of == e].T for e in range(n_experts)])
    size = np.stack([np.abs(a[:, of == e]) @ np.abs(b[:, of == e]).T for e in range(n_experts)])
    return out, size
