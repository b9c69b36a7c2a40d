// kv4_attn.cu -- attention over the 4-bit key/value cache: which kernel takes which sequences.
//
// Sequences with few query rows (tokens x heads that share a key/value head) are bound by the cache's
// bytes and go to kv4_decode.cu, longer ones by the products and go to kv4_prompt.cu. The lengths are
// on the device, so the host goes by the batch's bounds and launches the kernels that may be needed;
// each takes its own sequences and leaves the others. Measured, us, few-row and prompt kernel, at 4000 cached
// tokens a sequence: 16 x 16 rows of 5 heads x 128 30.1, 63.4; 16 x 32 rows 39.8, 64.4; 64 x 32 rows 110, 175;
// 1 x 32 rows 14.6, 18.6; 64 x 24 rows of 8 heads x 64 128, 184.
#include "kv4.cuh"

namespace bitnet {
namespace {

// The rows of a sequence that the few-row kernel takes, 0 if it is not needed: a batch of equal, longer
// sequences has none for it. Beside longer sequences it takes the single tokens, which make up most of such
// batches, with the instance for 8 rows (three blocks an SM) where they have no more; drafted tokens of more
// rows then go with the prompts (which of the two serves them better there was not measured). The instance for 16
// rows takes up to 32 as two units, so beside longer sequences 32 is the bound that both kernels are told.
int decode_rows(const Kv4& c, int share) {
  const int64_t all = (int64_t)c.max_q * share;
  if (all > kKvDecodeRows && (c.batch == 1 || (int64_t)c.batch * c.max_q == c.total_q)) return 0;
  if (all > kKvDecodeRows) return share <= 8 ? 8 : share <= kKvDecodeRows ? kKvDecodeRows : 0;
  return all <= 8 ? 8 : all <= 16 ? 16 : kKvDecodeRows;
}
int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

}  // namespace

int64_t kv4_attention_ws_bytes(const Kv4& c, int dim, int q_heads) {
  const int share = q_heads / c.kv_heads, rows = decode_rows(c, share);
  int64_t n = rows ? align256(kv4_decode_ws_bytes(c, dim, rows)) : 0;
  if ((int64_t)c.max_q * share > rows) n += kv4_prompt_ws_bytes(c, dim, share);
  return n;
}

cudaError_t launch_kv4_attention(const Kv4& c, int dim, const Kv4Attn& a, void* workspace, int num_sms,
                                 cudaStream_t st) {
  const int rows = decode_rows(c, a.share);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (rows) {
    if (cudaError_t e = launch_kv4_decode(c, dim, a, rows, ws, num_sms, st)) return e;
    ws += align256(kv4_decode_ws_bytes(c, dim, rows));
  }
  if ((int64_t)c.max_q * a.share <= rows) return cudaSuccess;
  return launch_kv4_prompt(c, dim, a, rows, ws, st);
}

}  // namespace bitnet
