// The lists that the chunk attention keeps in the caller's workspace between its kernels, and what an
// entry has to satisfy before anything is read or written by it.  The kernels of a call write the
// lists and read them back; a workspace that was given up, or handed to another call, too early holds
// something else by then.  Plain C++, so that the checks can be run on the host.
#pragma once

#ifdef __CUDACC__
#define COSA_HD __host__ __device__ __forceinline__
#else
#define COSA_HD inline
#endif

namespace cosa {

// one tile (pair) of the plan
struct ChunkTile {
  int tok0;  // first row of q
  int ntok;
  int pos0;  // cache position of that token
  int b;
  int jb, nb;  // key blocks, nb >= 1
  int kv;
  int prefix;
};
static_assert(sizeof(ChunkTile) == 32, "read as two 16-byte words");

// one row of the join list: the CTA whose share starts a tile that it does not finish
struct ChunkJoin {
  int ntok;  // 0: none
  int tok0, hk, pad0;
  int last;  // the CTA that finishes it
  int pad1[3];
};
static_assert(sizeof(ChunkJoin) == 32, "read as two 16-byte words");

// what the call's sizes allow
struct ChunkBounds {
  int batch, total_q, max_kv, num_kv_heads;
  int span;       // tokens a tile (pair)
  int max_tiles;  // room in the workspace
  int ctas;
};

// Units of work that a tile counts for besides its blocks (its Q load, its epilogue): without
// them the shares that get many short tiles end last.  Packed documents of 1,500 tokens, for
// 0, 1, 2, 3, 4 units: 247, 221, 199, 202, 215 us.
constexpr int CHUNK_SETUP = 2;

COSA_HD int chunk_blocks(int kv) { return (int)(((long long)kv + 127) >> 7); }

COSA_HD bool rows_fit(const ChunkBounds& n, int tok0, int ntok) {
  return ntok >= 1 && ntok <= n.span && tok0 >= 0 && tok0 <= n.total_q - ntok;
}

// number of tiles, and units of work of one head
COSA_HD bool plan_fits(const ChunkBounds& n, int tiles, long long units) {
  return tiles >= 0 && tiles <= n.max_tiles && units >= 0 &&
         units <= (long long)tiles * (chunk_blocks(n.max_kv) + CHUNK_SETUP);
}

// a tile that a share meets `at` units behind the tile's start
COSA_HD bool tile_fits(const ChunkBounds& n, const ChunkTile& t, long long at, int hk) {
  return rows_fit(n, t.tok0, t.ntok) && t.b >= 0 && t.b < n.batch && t.kv >= 1 && t.kv <= n.max_kv &&
         t.jb >= 0 && t.nb >= 1 && t.nb <= chunk_blocks(t.kv) - t.jb && at >= 0 &&
         at < (long long)t.nb + CHUNK_SETUP && hk >= 0 && hk < n.num_kv_heads;
}

// the entry of CTA `first`, whose ntok is not 0
COSA_HD bool join_fits(const ChunkBounds& n, int ntok, int tok0, int hk, int first, int last) {
  return rows_fit(n, tok0, ntok) && hk >= 0 && hk < n.num_kv_heads && last > first && last < n.ctas;
}

// The walk of one CTA of the single-token form over its share: `left` blocks from block `off` of
// sequence b's tile on.  It has no list: tile_of(b) works a sequence's tile out from the lengths each time
// (nb = 0: no tokens).  Lengths that are changed while the kernel runs must not keep it from
// ending, nor take it outside: where the blocks that the share was cut from are no longer there the
// walk is over, and `lost` set.
struct DecodeWalk {
  long long left;
  int b, hk, off;
  ChunkTile tile;
  int jb, nb, part;
  bool have;  // tile is that of b
  bool lost;

  template <typename TileOf>
  COSA_HD bool next(int batch, int num_kv_heads, const TileOf& tile_of) {
    if (left <= 0) return false;
    while (!have && hk < num_kv_heads) {  // sequences without tokens have no blocks
      tile = tile_of(b);
      have = tile.nb > 0;
      if (!have && ++b == batch) {
        b = 0;
        ++hk;
      }
    }
    const int rest = tile.nb - off;
    if (!have || rest <= 0) {
      lost = true;
      left = 0;
      return false;
    }
    jb = tile.jb + off;
    nb = left < rest ? (int)left : rest;
    part = off > 0 ? 0 : (nb < tile.nb ? 1 : -1);
    return true;
  }
  COSA_HD void advance(int batch) {
    left -= nb;
    off = 0;
    have = false;
    if (++b == batch) {
      b = 0;
      ++hk;
    }
  }
};

}  // namespace cosa
