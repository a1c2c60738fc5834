// dsa_kv4_span.h -- the notes an attention call's CTAs leave for the kernel
// that joins their partial results.
#pragma once

#ifdef __CUDACC__
#define DSA_HOST_DEVICE __host__ __device__
#else
#define DSA_HOST_DEVICE
#endif

namespace dsa {

// Whether a note names results of this call's `ctas` CTAs: `n` of them from
// `cta` on, the first one's result number `which` of its two.  A CTA whose wait
// gave up leaves its notes unwritten, and the workspace is whatever the caller's
// memory held.
DSA_HOST_DEVICE inline bool span_noted(int cta, int n, int which, int ctas) {
  return cta >= 0 && cta < ctas && n >= 1 && n <= ctas - cta && (which == 0 || which == 1);
}

}  // namespace dsa
