// Shared by the host entry points (wfst_score_api.cpp) and the gfx950 kernels
// (wfst_layer*.hip, wfst_adapters.hip, wfst_norm.hip, wfst_sample.hip, wfst_tokens.hip)
// of the operators around the search: the output layer with 4-bit weights and the
// low-rank adapters beside it, the log-softmax, the draw of tokens and the scores of
// given tokens. Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

namespace wfst {

// Host helpers of wfst_api.cpp: record the calling thread's error message and
// return `code`; check a caller's device buffer (see there).
int api_fail(int code, const std::string &msg);
int api_check_buffer(const void *p, size_t bytes, int device, const char *what, const char **lo = nullptr,
                     const char **hi = nullptr);

// Element types (the public WFST_LP_* values).
enum : int32_t { kF32 = 0, kF16 = 1, kBF16 = 2 };

inline size_t dtype_size(int32_t t) { return t == kF32 ? 4 : 2; }

// Rows of a padded [B, T] batch: row r = b * T + t holds data iff t < lengths[b]
// (every row when lengths is null). Rows without data are neither read nor written.
struct RowSet {
    const int32_t *lengths;
    int32_t T;
};

// ---- output layer

constexpr int kTileN = 16;      // output features of one weight tile
constexpr int kTileK = 128;     // input features of one weight tile

// A layer's device arrays. Weight tile (n / 16, k / 128) is 1024 bytes: 16 bytes
// for each of 64 lanes; lane l holds output feature l % 16, and its word j the
// features k = 32 j + 8 (l / 16) .. + 7 of the tile, feature 2p in bits 4p .. 4p+3
// and feature 2p + 1 in bits 16+4p .. 16+4p+3 (the order in which a shift and a
// mask yield the two halves of one register). Scales and zeros come gpt to a tile
// and feature, [n / 16][k / 128][n % 16][gpt]: 1 where groups are multiples of
// 128 features (a scale is repeated in each of its group's tiles), 2 for groups
// of 64, 4 (every 32 features) for all others.
struct Layer {
    const uint4 *w;
    const void *scales;         // binary32, or 16 bits as the caller gave them
    const uint8_t *zeros;       // null: 8
    const float *bias;          // null: 0
    int32_t K, N, group, gpt, kb, nt;
    int32_t scale_dtype;
};

struct LayerSource {
    const uint8_t *w;           // [N, ceil(K / 2)], feature 2i in the low half of byte i
    const void *scales;         // [N, ceil(K / group)]
    const uint8_t *zeros;       // the same shape, or null
    const float *bias;          // [N] or null
};

// Low-rank adapters of one layer, slots of them, each down [rank, K] and up [N, rank]
// of an own rank (0: none) and scale. A slot's down is [rb * 16][kp], features past K
// 0; its up holds for feature tile nt (16 of them) and 16 ranks jb 4 elements for each
// of 64 lanes, [nt][rb][64][4]: lane l has feature l % 16 and ranks 16 jb + 4 (l / 16)
// .. + 3, 0 past the slot's rank.
struct Adapters {
    void *down, *up;
    float *scales;              // [slots]
    int32_t *ranks;             // [slots]
    int32_t K, N, slots, rank;  // rank: the largest
    int32_t rb, kp, nt, dtype;
};

struct AdapterSource {
    const void *down, *up;
    int64_t down_stride, up_stride;
    int32_t rank;
    float scale;
};

// Row r of a call takes the adapter ids[r / per_id], none where that is no slot.
struct AdaptCall {
    Adapters a;
    const int32_t *ids;         // null: no adapters
    int32_t per_id;
    char *h;                    // blocks of 16 rows and 16 ranks, [rows / 16][rb], in the workspace
    uint4 *lists;               // [rows / group][parts][group * rb], there too
    int32_t *counts;            // [rows / group][parts]
    int32_t group, parts;       // rows whose blocks are listed together, and lists for them (set by the launch)
};

hipError_t launch_adapters_clear(const Adapters &a, hipStream_t s);
hipError_t launch_adapter_load(const Adapters &a, int32_t slot, const AdapterSource &src, hipStream_t s);

struct LayerCall {
    const void *x;
    void *out;
    int64_t x_stride, out_stride;
    int32_t M;
    int32_t x_dtype, out_dtype;
    RowSet rows;
    void *workspace;            // layer_workspace bytes
    AdaptCall ad;
};

// Bytes of h, of the lists and of their lengths in a call's workspace.
struct AdaptBytes { size_t h, lists, counts; };
AdaptBytes adapt_bytes(const Adapters &a, int32_t rows);
size_t layer_workspace(const Layer &l, int32_t rows, int32_t x_dtype);
hipError_t launch_layer_pack(const Layer &l, const LayerSource &src, uint4 *w, void *scales, uint8_t *zeros,
                             float *bias, hipStream_t s);
hipError_t launch_layer(const Layer &l, const LayerCall &c, hipStream_t s);
hipError_t launch_layer_f32(const Layer &l, const LayerCall &c, hipStream_t s);    // (by the type of x)
hipError_t launch_layer_f16(const Layer &l, const LayerCall &c, hipStream_t s);
hipError_t launch_layer_bf16(const Layer &l, const LayerCall &c, hipStream_t s);

// ---- log-softmax

struct NormCall {
    const void *x;
    void *out;
    const float *bias;          // [V] or null
    int64_t x_stride, out_stride, rows;
    int32_t V;
    int32_t x_dtype, out_dtype;
    float scale;
    RowSet set;
    void *workspace;            // norm_workspace bytes
};

int norm_pieces(int32_t V, int32_t x_dtype, int32_t out_dtype);
size_t norm_workspace(int64_t rows, int32_t V, int32_t x_dtype, int32_t out_dtype);
hipError_t launch_log_softmax(const NormCall &c, hipStream_t s);

// ---- draw

struct SampleCall {
    const void *x;
    int64_t x_stride, rows;
    int32_t V, x_dtype;
    const float *u;
    float temperature, top_p, min_p;
    int32_t top_k;
    const float *temperatures, *top_ps, *min_ps;   // one a row, or null
    const int32_t *top_ks;
    int32_t *token;
    float *log_prob;            // may be null
    int32_t *kept;              // may be null
    RowSet set;
    void *workspace;            // sample_workspace bytes
};

int sample_chunks(int64_t rows, int32_t V, int32_t x_dtype);
size_t sample_workspace(int64_t rows, int32_t V, int32_t x_dtype);

hipError_t launch_sample(const SampleCall &c, hipStream_t s);

// ---- scores of given tokens

constexpr int kMaxTokens = 256; // given tokens of one row
constexpr int kMaxTop = 64;     // alternatives of one row

struct TokenCall {
    const void *x;
    int64_t x_stride, rows;
    int32_t V, x_dtype;
    const int32_t *tokens;      // [rows, C]
    int32_t C, top_n;
    float temperature;
    const float *temperatures;  // one a row, or null
    float unit, scale;          // a power of two and log2 e / (unit temperature) (set by the launch)
    float *log_probs;           // [rows, C]
    int32_t *ranks;             // [rows, C]
    float *entropies;           // [rows] or null
    int32_t *top_tokens;        // [rows, top_n]
    float *top_log_probs;       // [rows, top_n]
    RowSet set;
    void *workspace;            // token_workspace bytes
};

size_t token_workspace(int64_t rows, int32_t V, int32_t C, int32_t top_n, int32_t x_dtype);

hipError_t launch_token_scores(const TokenCall &c, hipStream_t s);

}  // namespace wfst
