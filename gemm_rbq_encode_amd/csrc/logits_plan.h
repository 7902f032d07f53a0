// logits_plan.h -- how the rows of logits are cut over workgroups.  Host
// arithmetic only, so that a test can ask it without a GPU.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace rbq {

constexpr int LG_THREADS = 512;      // threads of a workgroup on a long row
constexpr int LG_VEC = 8;            // consecutive logits a thread takes at a time
constexpr int LG_SLICES_MAX = 256;   // slices of a row

constexpr int LG_TOPS = 1 << 14;     // vectors of a slice whose maxima LDS holds

// Slices of a row.  Cutting takes a second launch and a second start of every
// workgroup, so only a few long rows are cut, each thread with one vector at least.
// us whole / cut, fp16 (before rows were held in LDS and the named tokens' shares read
// eight at a time, which takes 4 us off a distillation step on either side):
//              sums alone    20 alternatives    gradient      distillation and gradient
//   1 x  32000   5.2   5.7      11.1  12.9       7.8   7.6       11.1  11.2
//  64 x  32000   6.4   7.7      13.6  15.4       9.2   9.8       12.9  13.9
//   1 x  64000   7.3   5.7      14.8  13.4      11.7   7.6       15.1  10.9
//  64 x  64000   9.0   8.1      18.0  16.7      13.5  10.4       17.1  14.3
// 256 x  64000  11.0  13.7      20.3  22.2      17.7  21.6       21.9  26.5
//   1 x 128256  11.9   5.7      19.0  14.8      19.9   7.9       23.5  11.3
//  64 x 128256  13.9   9.5      22.8  18.8      21.5  13.4       25.6  17.4
// 128 x 128256  15.2  13.6      24.1  22.2      24.1  21.5       28.4  25.8
// 256 x 128256  17.3  19.4      26.0  28.6      33.5  38.3       37.0  43.9
inline int logits_slices(int M, int vocab) {
    const int64_t vectors = ((int64_t)vocab + LG_VEC - 1) / LG_VEC;
    if (vectors < 6000 || M > vectors / 100)
        return 1;
    const int64_t want = std::min<int64_t>((1024 + (int64_t)M - 1) / M, LG_SLICES_MAX);
    const int64_t most = (vectors + LG_THREADS - 1) / LG_THREADS;
    return (int)std::max<int64_t>(1, std::min(want, most));
}

// Threads of a workgroup on slices of `each` vectors, with k alternatives.  More
// wait longer for each other at every step of a short row, and share the steps of
// a long one.  us with 512, 256 and 128 threads, 64 million fp16 logits in rows of
//                       1000            4000           16000           32000          128256 (2048 rows)
//   sums alone      176  103   66    66   42   35    34   31   32    29   30   29     96   97
//   gradient        234  135   86    85   63   58    57   62   67    61   65   64    247  254
//   distillation    543  287  216   171  114  100    89   78   83    74   78   80    257  278
// (with parts of the rows held in LDS since: gradient 86, 52, 55 with 128, 256 and 512
// threads on rows of 1000, 4000 and 32000, distillation 88 and 63 on 4000 and 32000)
//   64 alternatives 750  346  229   208  109   91    76   51   53    54   44   51    118  135
// More than 64 alternatives need more threads than they are.
inline int logits_threads(int each, int k) {
    if (k > 0)
        return each > 12000 ? 512 : each > 1200 || k > 64 ? 256 : 128;
    return each > 1800 ? 512 : each > 900 ? 256 : 128;
}

// Bytes of the partial results of all slices, 0 where a row is one slice: per
// slice a running maximum, two sums and the target's logit, and `top` keys of 8
// bytes; per row the logits of `slots` named tokens.
inline size_t logits_workspace_bytes(int M, int vocab, int top, int slots) {
    const int S = logits_slices(M, vocab);
    return S == 1 ? 0 : (size_t)M * ((size_t)S * (16u + 8u * (size_t)top) + 4u * (size_t)slots);
}

}  // namespace rbq
