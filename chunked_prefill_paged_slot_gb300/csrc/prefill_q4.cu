// prefill_q4.cu -- the chunk kernel over the 4-bit cache: prefill_tc.cu's, compiled in a
// translation unit of its own so that the two build side by side.
#define CPSA_CHUNK_Q4
#include "prefill_tc.cu"
