// Device helpers of the attention of several new tokens per stream.
#pragma once

#include "extend.h"
#include "kdecode.h"

namespace convt {

// A stream's cached tokens within what the call handles.
__device__ __forceinline__ int cut_length(const ExtendArgs &a, int b) {
    const int len = a.lengths[b];
    return len < 0 ? 0 : len > a.max_length ? a.max_length : len;
}

// starts[b] within the rows there are.
__device__ __forceinline__ int cut_start(const ExtendArgs &a, int b) {
    const int s = a.starts[b];
    return s < 0 ? 0 : s > a.tokens ? a.tokens : s;
}

// The stream that row `token` of q belongs to and the end of its rows; -1 for
// a row of no stream. starts does not decrease, so the first stream that ends
// behind the row is found by halving; values that do decrease give some stream
// or none.
__device__ __forceinline__ int stream_of(const ExtendArgs &a, int token, int &end) {
    if (!a.starts) {
        end = token + 1;
        return token;
    }
    int lo = 0, hi = a.batch;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.starts[mid + 1] > token) hi = mid;
        else lo = mid + 1;
    }
    if (lo == a.batch || a.starts[lo] > token) return -1;
    end = a.starts[lo + 1];
    return lo;
}

}  // namespace convt
