// mq_kv_join.h -- the record of a row pass of attention whose partials several workers hold, and what makes one safe to follow (plain C++:
// the tests compile it for the host).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MQ_HD __host__ __device__ __forceinline__
#else
#define MQ_HD inline
#endif

namespace mq {

// a row pass that began with a worker and ends with another: its partials are number 1 of workers first .. last - 1 and number 0 of the last
struct AtJoin {
    int32_t nrow, last, h, r0;      // nrow 0: none
    int64_t tok;
};

// Whether worker `first`'s record names workers that there are and rows of this call.  Every worker writes its record (nrow 0) before its
// first wait, so that this holds even where a wait has run out; the join follows no record for which it does not.
MQ_HD bool at_join_holds(const AtJoin &w, int32_t first, int32_t workers, int32_t rows, int32_t H, int32_t group, int64_t n_tokens) {
    return w.nrow > 0 && w.nrow <= rows && w.last > first && w.last < workers && w.h >= 0 && w.h < H && w.r0 >= 0 && w.tok >= 0 &&
           w.tok < n_tokens && ((int64_t)w.r0 + w.nrow - 1) / group < n_tokens - w.tok;
}

}  // namespace mq
