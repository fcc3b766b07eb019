// Block cache: many-query attention with prefixes (kvarn_block_prefill.cu).
#define KVARN_BLOCK_MORE 1
#include "kvarn_block_prefill.cu"
