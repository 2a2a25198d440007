// The paged attention kernels whose scores are capped by a tanh or biased by the
// distance: a translation unit of their own, compiled beside the plain ones.
#define PA_SCORED
#include "paged_attention.cu"
