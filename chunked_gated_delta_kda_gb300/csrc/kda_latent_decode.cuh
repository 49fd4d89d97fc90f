// Parameters of the absorbed (decode) form.
#pragma once

#include "kda_latent.cuh"

namespace kda {

struct DecodeParams {
    const void* q;              // [N, S, H, 576]
    const void* cache;          // [num_pages * page_size, 576]
    const int32_t* table;       // [N, table_width]
    const int32_t* lens;        // [N]
    void* o;                    // [N, S, H, 512]
    float* lse;                 // [N, S, H] or null
    uint8_t* workspace;
    uint32_t* status;
    float scale;
    int num_pages, page_size, table_width;
    int N, S, H;
    uint32_t wait_limit;
};

constexpr int DEC_CTAS = 152;   // one a SM

struct DecodeScratch {
    uint32_t* err;              // [DEC_CTAS] status bits
    long long* prefix;          // [N + 1] 64-key tiles before each sequence
    float* lse;                 // [2 DEC_CTAS][rows of a unit]
    float* o;                   // [2 DEC_CTAS][rows of a unit][512]
};

}  // namespace kda
