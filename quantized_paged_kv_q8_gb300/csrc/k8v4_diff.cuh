// What the kernels of differential attention share: the layout of their partial rows
// and the combine that joins them.
#pragma once

#include "k8v4_ops.cuh"

namespace k8v4 {

// A partial row: o[256] (rotated space, unnormalised, relative to 2^m), m (a base-2
// exponent, -inf: no cell seen), l (the sum of 2^(score - m)), two unused floats.
constexpr int kDiffRow = 260;

// Where the partial rows of a (row, KV head) are: split s of map m and query head h (of the
// head's 8) at ws + (((first + s) * 2 + m) * 8 + h) * kDiffRow.
// The rows of single queries: first = (row * H + g) * splits, all with `splits` splits.
int launch_diff_combine(const Launch& L, const float* ws, int splits, const int32_t* row_seq, int n_rows, int H,
                        const k8v4_diff& diff, void* out);

}  // namespace k8v4
