// Block cache: decode attention with prefixes and weights (kvarn_block_decode.cu).
#define KVARN_BLOCK_MORE 1
#include "kvarn_block_decode.cu"
