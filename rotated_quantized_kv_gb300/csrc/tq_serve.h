// tq_serve.h -- private declarations of the serving calls (rotary positions,
// ragged writes and reads, tree attention): kernel parameters and launchers.
#pragma once

#include "tq_internal.h"

namespace tqk {

// ----------------------------------------------------------------- rotary positions
struct RopeTable {               // tq_rope_table
    double freq[TQ_MAX_HEAD_DIM / 2];
    double amplitude;
    int half, first, n;
    float *table;
};

struct RopeView {
    const float *table;          // [n_pos][2][half], or nullptr: no rotary positions
    int half, interleaved, n_pos;
};

struct RopeTensorParams {
    const void *in;
    void *out;
    int64_t is[3], os[3];        // strides of (b, h, t)
    int head0;                   // first head in the concatenation of the call's tensors
};

struct RopeParams {
    RopeView rope;
    const int *positions;
    int64_t pos_stride;
    int B, T, d, inverse;
    int n_tensors, heads;        // heads: over all tensors
    RopeTensorParams x[TQ_MAX_ROPE_TENSORS];
};
cudaError_t launch_rope_table(const RopeTable &p, cudaStream_t s);
cudaError_t launch_rope(const RopeParams &p, int dtype, cudaStream_t s);

// ----------------------------------------------------------------- segments
// A segment as the serving kernels address it: rows of (b, h, t).
struct SegView {
    int fp16;                    // fp16 segment: k, v are its rows
    int capacity;
    const uint8_t *k, *v;        // packed codes (or fp16 rows) of (0, 0, 0)
    const float *ks, *vs;        // packed: scales of (0, 0, 0)
    uint64_t kblock, vblock;     // bytes per batch element
    uint64_t koff[kMaxH], voff[kMaxH];  // byte offset of a head inside a batch block
    uint8_t kbits[kMaxH], vbits[kMaxH];
};

struct RowMap {                  // rows of a ragged write or read
    const int *t_begin, *n_rows; // n_rows: nullptr: n_max
    const int *index;            // source row of row j (writes), or nullptr
    int64_t index_stride;
    int n_max, n_source;
};

struct AppendParams {
    SegView seg;
    RowMap rows;
    RopeView rope;
    const int *positions;
    int64_t pos_stride;
    const uint16_t *K, *V;
    int64_t ks[3], vs[3];        // strides of (b, h, s)
    int B, H, d;
    uint32_t sign_bits[kMaxD / 32];
    float inv_sqrt_d;
    float thr[kCbTotal];         // value thresholds, flat by bit width
    int law;
    uint32_t vwidths;            // bit b: some head's values have b bits
    int vec;                     // 8-byte loads of the source
};
cudaError_t launch_append(const AppendParams &p, cudaStream_t s);

// One thread per vector (head_dim 128), a launch per key and per value width: r.X,
// its strides and r.T (rows a sequence may get) describe the source rows.
struct AppendRowsParams {
    RowsParams r;
    RowMap rows;
    RopeView rope;               // keys
    const int *positions;
    int64_t pos_stride;
};
cudaError_t launch_append_keys(const AppendRowsParams &p, int bits, bool beside, cudaStream_t s);
cudaError_t launch_append_values(const AppendRowsParams &p, int bits, bool beside, cudaStream_t s);

struct ReadParams {
    SegView seg;
    RowMap rows;
    void *K, *V;                 // either may be null
    int64_t ks[3], vs[3];
    int B, H, d;
    int rotate;                  // apply R
    uint32_t sign_bits[kMaxD / 32];
    float inv_sqrt_d;
    float centroid[kCbTotal];
    uint32_t vwidths;            // bit b: some head's values have b bits
    int vec;                     // stores of four coordinates
};
cudaError_t launch_read(const ReadParams &p, int dtype, cudaStream_t s);

// One thread per vector of head_dim 128 or two of 64, a launch per key and per value width.
struct ReadRowsParams {
    RowMap rows;
    const uint8_t *codes;
    const float *scale;
    uint64_t block, off[kMaxH];
    int B, H, capacity, n_heads; // heads of this launch
    uint8_t head[kMaxH];
    void *out;
    int64_t st[3];
    int dtype, vec, rotate;      // vec: 16-byte stores
    uint32_t flip[32];           // record words: ones in the fields of the coordinates to negate
    float out_scale[kD];         // coordinates m and m + 64 of a thread's 128
    float level[256];            // values: the centroids
};
cudaError_t launch_read_keys(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s);
cudaError_t launch_read_values(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s);
cudaError_t launch_read_keys_d64(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s);
cudaError_t launch_read_values_d64(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s);

// ----------------------------------------------------------------- tree attention
// The work is a list of 128-token tiles.  For sequence b in order, KV head h,
// block of query rows rb (of R rows; row = draft * g + query head of the group):
// the tiles of b's packed segments, then those of its fp16 segments.  The workers
// take contiguous ranges of the list, all of the same length but the last.  The tiles of one (b, h, rb) are cut
// into parts: packed tiles every kTreePart, the fp16 ones likewise; every worker
// leaves one record (m, l, sum per row) for each part that it touches, at slot
// worker + part index (the pairs (worker, part) form a monotone path, so that
// the sums are distinct).  The merge adds the drafted tokens.
constexpr int kTreeTile = 128;
constexpr int kTreePart = 128;   // tiles: bounds the length of one tensor-core sum

struct TreeSeg {
    SegView seg;
    const int *len;              // per-sequence length or nullptr
    int n_tokens;
    int law;                     // value codebook
};

// What the merge needs of it: the list's geometry without the segments' data.
struct TreeListSeg {
    const int *len;
    int n_tokens;
};
struct TreeList {
    int B, H, g, N, R, n_rb;
    int n_seg, n_packed, ragged;
    int parts_packed, parts, workers;
    TreeListSeg seg[TQ_MAX_SEGMENTS];
};
struct TreeQueryParams {
    int H, g, n_rb, n_var, rows;  // rows: N g
    const uint16_t *q;
    int64_t qs[3];
    uint8_t *images;
    int *error;
    uint8_t var_bits[TQ_MAX_SEGMENTS][kMaxH];
    uint32_t sign_bits[4];       // (head_dim 64 and 128)
    float inv_sqrt_d, qk_scale;
};
struct TreeMergeParams {
    TreeList t;
    const uint16_t *q, *k, *v;
    int64_t qs[3], ks[3], vs[3];
    const uint32_t *mask;
    int64_t mask_stride;
    int mask_words;
    uint16_t *out;
    const float *part;
    uint32_t sign_bits[kMaxD / 32];
    float inv_sqrt_d, qk_scale;
    int vec;                     // wide loads of q, k and v
};

struct TreeParams {
    int B, H, g, N, d, R, n_rb;  // g query heads per KV head, R rows per block, n_rb blocks
    int n_seg;                   // packed segments first
    int n_packed;
    int ragged;                  // some segment has per-sequence lengths
    int parts_packed, parts;     // parts per (b, h, rb): packed ones, all
    TreeSeg seg[TQ_MAX_SEGMENTS];
    const uint16_t *q, *k, *v;
    int64_t qs[3], ks[3], vs[3];
    const uint32_t *mask;
    int64_t mask_stride;
    int mask_words;
    uint16_t *out;
    float *part;                 // records: [slot][R][d + 4]: m (log2 units; any reference, the same for l and sum), l, pad, pad, sum
    // tensor-core form: the query blocks as MMA operands, one image per (b, h, rb) and
    // key width among the head's segments
    uint8_t *images;
    int n_var;
    uint8_t var[TQ_MAX_SEGMENTS][kMaxH];     // image of a segment
    uint8_t var_bits[TQ_MAX_SEGMENTS][kMaxH];  // key bits of image v (0: fp16 keys)
    int *error;
    int workers, wait_polls;
    uint32_t sign_bits[kMaxD / 32];
    float inv_sqrt_d, qk_scale;  // qk_scale: log2(e) / sqrt(d)
    float centroid[2][kCbTotal]; // by law
};
// Rows per block, workers and the kernel's choice for a shape: the same rule
// sizes the workspace and launches the kernel.
struct TreeShape {
    int R, n_rb, workers;
};
// Value levels of the tensor-core form: fp16(s c_k) by law, flat by width, and 1/s.
struct TreeLevels {
    uint16_t half[2][kCbTotal];
    float inv[2][9];
};
// Whether a head dimension takes the tensor-core form (64 and 128).
inline bool tree_on_tensor_cores(int d) { return d == 64 || d == 128; }
cudaError_t launch_tree_mma(const TreeParams &p, cudaStream_t s);
// Bytes of a query image: hi and lo parts (rows of d fp16), 32 bytes a row for the
// constants' step, and the factor A.
inline size_t tree_image_bytes(int d, int R) { return (static_cast<size_t>(4) * d * R + 32 * R + 16 + 127) / 128 * 128; }
int tree_mma_rows(int rows);
TreeShape tree_shape(int B, int H, int g, int N, int d, long long tiles_per_head);
cudaError_t launch_tree(const TreeParams &p, cudaStream_t s);

// ----------------------------------------------------------------- from tq_host.cpp
tq_status layout_status(const tq_segment_layout *L, bool need_bits);
void value_thresholds(float *flat, const uint8_t *bits, int H, int law);
void value_centroids(float *flat, const uint8_t *bits, int H, int law);
float rotation_scale(int d);
int decode_wait_polls();
int current_sm_count();
void fill_rows_rotation(RowsParams &p, const uint32_t *sign_bits, int d);
bool fill_rows_values(RowsParams &p, int bits, int law);

}  // namespace tqk
