// Launch interface between the C-ABI layer (api_attention.cu) and the kernels
// of attention to other states (include/convrot_block.h).
#pragma once

#include "../csrc/block.h"

namespace convrot {

// A tensor [batch, tokens, heads, d] of 16-bit elements whose heads start on 16
// bytes, as the kernels' copies read it. Strides in elements: batch, token, head.
struct States {
    const void *p;
    int64_t tokens, heads;
    int64_t strides[3];
};

constexpr int kTileKeys = 128;

// Rows of a gathered sample: whole tiles.
inline int64_t gathered_rows(int64_t tokens) { return (tokens + kTileKeys - 1) / kTileKeys * kTileKeys; }

// Copies the heads of `count` tensors (1, or keys and values) to [batch, rows, heads, dp], dp = d rounded up to 8. Without a
// mask, rows = tokens. With one, rows = gathered_rows(tokens): the tokens that are there come first, in order, zeros follow
// to the end of the last tile that has one; counts[b] is their number and index[b * rows + i] the token of row i; and
// rows of zero[i] (dense [batch, tokens, heads, d]) at tokens that are not there become zero.
struct GatherArgs {
    const void *src[2];
    int64_t strides[2][3];
    void *dst[2];
    void *zero[2];
    int32_t count;
    const uint8_t *mask;
    int64_t mask_stride;
    int32_t *counts, *index;
    int64_t batch, tokens, heads, rows;
    int32_t d, dp;
};
cudaError_t launch_gather(const GatherArgs &a, cudaStream_t stream);

// Masks of one tile's keys are applied where they are (the gathering kernel's 5 us are more than what a shorter tile saves),
// longer ones by gathering the keys that are there (3 samples of 1363 queries, 24 heads, a third to all of 333 keys: 22 us with
// it against 28 over all tiles). A mask of no keys is none: where it is applied, each item has its tile.
inline bool mask_in_place(int64_t kv_tokens) { return kv_tokens > 0 && kv_tokens <= kTileKeys; }

struct AttentionArgs {
    States q, k, v;
    const int32_t *counts;  // keys of each sample, or null: k.tokens
    const uint8_t *mask;    // of at most kTileKeys keys, where it is to be applied in place; else null
    int64_t mask_stride;
    void *out;
    int64_t out_strides[3];
    float *lse;
    int32_t *dev_status;
    int64_t batch;
    int64_t kv_tokens;      // at most
    float scale;
    int32_t d, dtype;
    int32_t splits;         // shares of the keys, each with items of its own: attention_splits
    float *partial;         // attention_partial_bytes, where there are several
};
cudaError_t launch_attention(const AttentionArgs &a, cudaStream_t stream);
// Shares of the keys, where the items (some queries of a head each) are few and the keys long: as many as the SMs take at once,
// if that saves an item six tiles of keys or more, since the second kernel that puts the shares together costs as much as about
// five (16 items of 64 queries, 4096 keys: 38 -> 15 us; 64 items, 1000 keys: 12.6 us whole, 13.1 in two; 72 items, 600 keys:
// 11.4 and 14.8). A second kernel's warp has one lane a share.
inline int32_t key_shares(int64_t items, int64_t kv_tokens)
{
    const int64_t tiles = (kv_tokens + kTileKeys - 1) / kTileKeys;
    if (items == 0 || items > kSms / 2) return 1;
    int64_t shares = kSms / items < tiles / 2 ? kSms / items : tiles / 2;
    if (shares > 32) shares = 32;
    return shares > 1 && tiles - (tiles + shares - 1) / shares >= 6 ? static_cast<int32_t>(shares) : 1;
}
// A kernel's forms: all tiles of a head's keys pass by; one tile stays with a CTA; shares of the keys have items of their own.
// (A form each: the shares' arithmetic in the first one cost it 2 %.)
enum KeyForm { kPass, kStays, kShared };
int32_t attention_splits(int64_t batch, int64_t q_tokens, int64_t kv_tokens, int64_t q_heads);
int64_t attention_partial_bytes(int64_t batch, int64_t q_tokens, int64_t kv_tokens, int64_t q_heads, int d);

// Few queries: keys and values whose heads start on 16 bytes (queries may start anywhere), the mask read as it is.
bool attention_few_takes(int64_t q_tokens, int64_t q_heads, int64_t kv_heads);
int64_t attention_few_partial_bytes(int64_t batch, int64_t kv_tokens, int64_t kv_heads, int d);
cudaError_t launch_attention_few(const AttentionArgs &a, const uint8_t *mask, int64_t mask_stride, float *partial, cudaStream_t stream);

// Rows of each head's statistics in the backward pass: whole tiles of queries.
constexpr int kTileQueries = 128;
inline int64_t stat_rows(int64_t tokens) { return (tokens + kTileQueries - 1) / kTileQueries * kTileQueries; }
// Tokens of one block of the statistics (a block has one query head's): 64, and more where the heads that share a key head
// would have over 256 blocks together, since what follows takes the largest value of all of them.
inline int64_t stat_tokens(int64_t tokens, int64_t group) { return (stat_rows(tokens) * group + 64 * 256 - 1) / (64 * 256) * 64; }
inline int64_t stat_blocks(int64_t tokens, int64_t group) { return (stat_rows(tokens) + stat_tokens(tokens, group) - 1) / stat_tokens(tokens, group); }

struct AttentionGradArgs {
    States q, k, v, dout;     // as the kernels read them
    const int32_t *counts, *index;
    int64_t index_rows;       // of a sample in index
    const uint8_t *mask;      // as in AttentionArgs
    int64_t mask_stride;
    const void *out, *dout_own;
    int64_t out_strides[3], dout_own_strides[3];  // the caller's out and dout, for the statistics
    const float *lse;
    float *base2, *delta;     // [batch, q_heads, stat_rows]: -lse in base 2, and -dout . out
    float *amax;              // float16: [batch, kv_heads, q_heads / kv_heads, blocks] largest |dout|; else null
    float *partial;           // grad_kv_partial_bytes
    float *partial_q;         // grad_q_partial_bytes
    void *dq, *dk, *dv;
    int32_t *dev_status;
    int64_t batch, kv_tokens;
    float scale;
    int32_t d, dtype;
};
int64_t grad_kv_partial_bytes(int64_t batch, int64_t q_tokens, int64_t kv_tokens, int64_t q_heads, int64_t kv_heads, int d);
int64_t grad_q_partial_bytes(int64_t batch, int64_t q_tokens, int64_t kv_tokens, int64_t q_heads, int d);
// Whether launch_attention_grad_kv makes dq too.
bool grad_kv_makes_dq(int64_t kv_tokens, int d);
cudaError_t launch_attention_stats(const AttentionGradArgs &a, cudaStream_t stream);
cudaError_t launch_attention_grad_q(const AttentionGradArgs &a, cudaStream_t stream);
cudaError_t launch_attention_grad_kv(const AttentionGradArgs &a, cudaStream_t stream);

// Shared memory and tensor-memory columns of every launch form, for the check that no mix of blocks waits for columns.
int attention_shared(int form, int *columns);  // 0 past the last form
int attention_grad_q_shared(int form, int *columns);
int attention_grad_kv_shared(int form, int *columns);

}  // namespace convrot
